// mma_common.cuh -- building blocks of the decode kernels: the shared-memory
// layout of a page's key and value blocks, ldmatrix and mma.sync wrappers, and
// the layout of a split's partial state.
#pragma once

#include <stdint.h>

#include "polar_common.cuh"

namespace polar {

constexpr int kChunkBytes = kPage * kHeadDim * 2;      // one (page, K|V, head): 8 KB
constexpr int kStageBytes = 2 * kChunkBytes;           // K and V
constexpr int kPartialFloats = 72;                     // acc[64] + 6 stats + 2 pad

// Byte offset of logical 16-byte chunk c of row t inside a 128B-swizzled tile.
__device__ __forceinline__ uint32_t swz(int t, int c) {
    return static_cast<uint32_t>(t * 128 + ((c ^ (t & 7)) << 4));
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// d += A(16x16; a0/a2 row g of the lane, a1/a3 row g+8) * B(16x8), bf16 in,
// fp32 accumulate.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Keep the low / high bf16 half of x only if the corresponding token is valid.
__device__ __forceinline__ uint32_t mask_pair(uint32_t x, bool lo_ok, bool hi_ok) {
    return (lo_ok ? (x & 0xFFFFu) : 0u) | (hi_ok ? (x & 0xFFFF0000u) : 0u);
}

}  // namespace polar
