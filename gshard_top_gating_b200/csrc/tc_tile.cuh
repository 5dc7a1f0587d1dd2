// tc_tile.cuh -- pieces shared by the tensor-core GEMM kernels: the shared-memory matrix
// descriptor, the walk over a grouped GEMM's tiles, a 16-byte shared load.
#pragma once

#include "common.cuh"

namespace moe {

// Shared-memory matrix descriptor, 128-byte swizzle (tcgen05 format: version 1 at bit 46,
// layout type 2 = SWIZZLE_128B at bits 61-63).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// Walks this CTA's tiles in the global order (expert, n-tile, m-tile).
struct TileIter {
  const int* tile_pre;   // smem [E+1]: first tile of each expert
  const int* mtiles;     // smem [E]
  int E, NT, e;
  __device__ bool decode(int tile, int& ex, int& mt, int& nt) {
    if (tile >= tile_pre[E]) return false;
    while (tile >= tile_pre[e + 1]) ++e;
    const int local = tile - tile_pre[e];
    const int m_e = mtiles[e];
    nt = local / m_e;
    mt = local - nt * m_e;
    ex = e;
    return true;
  }
};

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

}  // namespace moe
