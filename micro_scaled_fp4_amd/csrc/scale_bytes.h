// Scale bytes of rows of any length and alignment, for the FP4 products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4dev {

constexpr int kBufferWord3 = 0x00020000;       // raw buffer descriptor word 3 (gfx9 family)
constexpr int kOutOfRange = 0x7ffffff0;        // a buffer offset past every range: reads 0

// Descriptor of `bytes` scale bytes from p on; ALIGNED false: of the aligned
// dwords that hold them, p at byte `lead` of the first.
struct ScaleRange {
  __amdgpu_buffer_rsrc_t rsrc;
  int lead;
};
template <bool ALIGNED>
__device__ __forceinline__ ScaleRange scale_range(const uint8_t* p, int bytes) {
  const int lead = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 3);
  const int n = ALIGNED || bytes <= 0 ? bytes : (bytes + lead + 3) & ~3;
  return {__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p) - lead, 0, n, kBufferWord3), lead};
}

// The DW dwords that start at byte `shift` (0..3) of s, zeroed from byte `valid` on.
template <int DW>
__device__ __forceinline__ void place_bytes(uint32_t (&out)[DW], const uint32_t (&s)[DW + 1], int shift,
                                            int valid) {
#pragma unroll
  for (int q = 0; q < DW; ++q) {
    const int v = valid - 4 * q;
    const uint32_t keep = v >= 4 ? ~0u : v <= 0 ? 0u : (1u << (8 * v)) - 1u;
    out[q] = __builtin_amdgcn_alignbyte(s[q + 1], s[q], shift) & keep;
  }
}

}  // namespace fp4dev
