// Parts that the tile kernels share: LDS DMA, waits, the order of tiles.
#pragma once
#include "common.hpp"

namespace ds4 {

// 64 lanes x 16 bytes from global memory into LDS at lds_dst + 16 * lane.
// Inline asm, so that the compiler's wait counts leave the LDS reads alone;
// the stage loop waits explicitly.
__device__ __forceinline__ void mt_dma16(const void* g, uint32_t lds_dst) {
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_dst);
    asm volatile(
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %0, off"
        :
        : "v"(g), "s"(m0)
        : "memory", "m0");
}

// Wait until at most N of this wave's vector-memory operations are outstanding.
template <int N>
__device__ __forceinline__ void mt_wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Workgroup barrier behind this wave's finished LDS reads.
__device__ __forceinline__ void mt_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Tile t of tr x tc tiles: groups of 8 row tiles, row tiles first inside a
// group, so that tiles that run together share operands in their L2.
__device__ __forceinline__ void mt_tile(int t, int tr, int tc, int& r, int& c) {
    const int sg = t / (8 * tc), rem = t - sg * (8 * tc);
    const int rows = min(8, tr - 8 * sg);
    c = rem / rows;
    r = 8 * sg + rem - c * rows;
}

}  // namespace ds4
