// attn_device.cuh - which keys of a paged cache a token sees, and tiled loads
// of its pages: shared by the decode and the prompt form of attention.
#pragma once

#include "block_device.cuh"

namespace w4 {

constexpr float kNegInf = -__builtin_huge_valf();

// Key j is visible to the token at position p.
__device__ __forceinline__ bool key_visible(int j, int p, int window, int sinks) {
    return j <= p && (window == 0 || p - j < window || j < sinks);
}

// The 16-key blocks that tokens p0 .. p1 (p0 <= p1) may see: blocks
// [0, ns) and [w0, we), listed as c = 0 .. n - 1.
struct KeyBlocks {
    int ns, w0, n;
    __device__ __forceinline__ int operator()(int c) const { return c < ns ? c : c - ns + w0; }
};

template <int BLK>
__device__ __forceinline__ KeyBlocks key_blocks(int p0, int p1, int window, int sinks) {
    KeyBlocks k{0, 0, 0};
    if (p1 < 0) return k;
    const int we = p1 / BLK + 1;
    // a window reaching back to key 0 hides nothing
    const int start = window > 0 && p0 >= window ? p0 - window + 1 : 0;
    k.w0 = start / BLK;
    k.ns = min((min(sinks, start) + BLK - 1) / BLK, k.w0);
    k.n = k.ns + we - k.w0;
    return k;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
           "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4),
           "r"(smem_u32(bar))
        : "memory");
}

}  // namespace w4
