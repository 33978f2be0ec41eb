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

// Transpose of an 8 x 8 matrix of 16-bit values: lane holds (row lane / 4,
// columns 2 (lane % 4) and + 1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// The lazy maximum of the one-token kernels, in log2 units: how far it may lag behind.
constexpr float kLazyOne = 8.f;

// One block of 16 keys for NT tiles of 8 query heads (attn_decode.cu describes the step): st, a stage
// [K: D / 64 panels of 16 rows, V the same]; qf, the lane's pieces of the queries; o, m, l and the
// offset -m sc, the running sums.  all: every key of the block, which starts at j0, is seen; else
// those that seen(j) says.
template <int D, int NT, typename Seen>
__device__ __forceinline__ void attend_block(const uint8_t* st, const uint4 (&qf)[NT][D / 32], float (&o)[NT][D / 16][4],
                                             float (&m)[NT][2], float (&l)[NT][2], float (&off)[NT][2], float sc, int j0,
                                             bool all, Seen seen) {
    const int lane = threadIdx.x & 31, ki = lane & 3, kj = lane >> 2, pj = (kj >> 1) + 4 * (kj & 1);
    // shared-memory offsets of the lane's pieces in a stage
    const uint32_t k_off = pj * 128 + ((ki ^ pj) << 4);                   // ^ 64: the panel's other half
    const uint32_t v_off = 16 * D * 2 + ki * 128 + ((pj ^ ki) << 4);      // n odd: ^ 64
    float s[NT][2][4];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[x][0][e] = s[x][1][e] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const uint8_t* kp = st + (c >> 1) * 2048 + (k_off ^ ((c & 1) * 64));
        const uint4 k0 = *reinterpret_cast<const uint4*>(kp), k1 = *reinterpret_cast<const uint4*>(kp + 1024);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            mma_bf16_16816(s[x][0], k0.x, k1.x, k0.y, k1.y, qf[x][c].x, qf[x][c].y, s[x][0]);
            mma_bf16_16816(s[x][1], k0.z, k1.z, k0.w, k1.w, qf[x][c].z, qf[x][c].w, s[x][1]);
        }
    }
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[x][0][e] += s[x][1][e];
    if (!all) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!seen(j0 + pj + 8 * (e >> 1))) s[x][0][e] = kNegInf;
    }
    bool grow = false;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) grow |= (fmaxf(s[x][0][e], s[x][0][e + 2]) - m[x][e]) * sc > kLazyOne;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(m[x][e], fmaxf(s[x][0][e], s[x][0][e + 2]));
#pragma unroll
                for (int z = 4; z < 32; z <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, z));
                // both -inf (nothing seen yet): the factor multiplies zeros
                const float f = mx == m[x][e] ? 1.f : ex2_approx((m[x][e] - mx) * sc);
                m[x][e] = mx;
                off[x][e] = mx == kNegInf ? 0.f : -mx * sc;
                l[x][e] *= f;
#pragma unroll
                for (int t = 0; t < D / 16; ++t) { o[x][t][e] *= f; o[x][t][e + 2] *= f; }
            }
    }
    uint32_t pb[NT][2], pl[NT][2];      // the weights' upper halves, and what they leave
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        float w0[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w0[e] = ex2_approx(fmaf(s[x][0][e], sc, off[x][e & 1]));
        l[x][0] += w0[0] + w0[2];
        l[x][1] += w0[1] + w0[3];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float u = w0[2 * h], v = w0[2 * h + 1];
            const uint32_t hi = prmt(__float_as_uint(u), __float_as_uint(v), 0x7632);
            pb[x][h] = movmatrix_trans(hi);
            // the factor keeps the rest of a bf16 weight above zero: 0 * inf is NaN
            constexpr float kUp = 1.f + 0x1p-23f;
            pl[x][h] = movmatrix_trans(pack_bf16x2(fmaf(u, kUp, -bf16x2_lo(hi)), fmaf(v, kUp, -bf16x2_hi(hi))));
        }
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        uint4 v[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            v[n] = *reinterpret_cast<const uint4*>(st + c * 2048 + n * 512 + (v_off ^ ((n & 1) * 64)));
            if (!all && !seen(j0 + ki + 4 * n)) v[n] = make_uint4(0, 0, 0, 0);
        }
        const uint32_t *v0 = &v[0].x, *v1 = &v[1].x, *v2 = &v[2].x, *v3 = &v[3].x;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t a0 = prmt(v0[t], v1[t], 0x5410), a1 = prmt(v0[t], v1[t], 0x7632);
            const uint32_t a2 = prmt(v2[t], v3[t], 0x5410), a3 = prmt(v2[t], v3[t], 0x7632);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                mma_bf16_16816(o[x][c * 4 + t], a0, a1, a2, a3, pb[x][0], pb[x][1], o[x][c * 4 + t]);
                mma_bf16_16816(o[x][c * 4 + t], a0, a1, a2, a3, pl[x][0], pl[x][1], o[x][c * 4 + t]);
            }
        }
    }
}

}  // namespace w4
