// attn_device.cuh - the warp-level core of attention over a paged cache:
// which keys a token sees, and one online-softmax step over 16 keys.
//
// A warp holds 16 query rows (rows r = lane / 4 and r + 8 of the mma.sync
// m16n8k16 layout) and takes 16 keys at a time.  Both products sum over an
// index whose order is free (the head dimension for q . k, the keys for
// p . v), so the fragments are chosen for the loads instead of the other way
// round: a lane's operand words are whole 16-byte pieces of key and value
// rows, copied straight from global memory, and no shared-memory transpose
// or ldmatrix is needed.
//   K piece (c, h): key lane / 4 + 8 h, values 32 c + 8 (lane % 4) .. + 7
//   V piece (c, n): key 2 (lane % 4) + (n & 1) + 8 (n >> 1), values
//                   64 c + 8 (lane / 4) .. + 7
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

template <int D>
struct Frag {                       // one step's K and V pieces of a lane
    uint4 k[D / 32][2];
    uint4 v[D / 64][4];
};

template <int D>
struct RowState {                   // of the lane's rows lane / 4 and lane / 4 + 8
    float o[D / 8][4];              // output accumulators (mma C layout)
    float m[2], l[2];               // running maximum of the raw scores; sum
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m[0] = m[1] = kNegInf;
        l[0] = l[1] = 0.f;
    }
};

// Output column of accumulator o[nt][e] (e & 1: second of its pair).
__device__ __forceinline__ int out_col(int nt, int e, int lane) {
    return (nt >> 3) * 64 + (2 * (lane & 3) + (e & 1)) * 8 + (nt & 7);
}

// One step: scores of 16 keys, running maximum, weights, sum, weighted values.
// vis[t][e]: key 8 t + 2 (lane % 4) + (e & 1) is visible to row e >> 1 of the
// lane's two.  qf: the query pieces of both rows; sc: softmax scale in units
// of log2.  l sums the fp32 weights; the weights are rounded to bf16 only as
// the matrix operand of the value product.
template <int D>
__device__ __forceinline__ void attn_step(RowState<D>& st, const uint4 (&qf)[D / 32][2],
                                          const Frag<D>& f, const bool (&vis)[2][4], float sc) {
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            mma_bf16_16816(s[t], qf[c][0].x, qf[c][1].x, qf[c][0].y, qf[c][1].y, f.k[c][t].x,
                           f.k[c][t].y, s[t]);
            mma_bf16_16816(s[t], qf[c][0].z, qf[c][1].z, qf[c][0].w, qf[c][1].w, f.k[c][t].z,
                           f.k[c][t].w, s[t]);
        }
    float mx[2] = {st.m[0], st.m[1]};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[t][e] = vis[t][e] ? s[t][e] : kNegInf;
            mx[e >> 1] = fmaxf(mx[e >> 1], s[t][e]);
        }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
    }
    if (__any_sync(0xffffffffu, mx[0] != st.m[0] || mx[1] != st.m[1])) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            // both -inf (nothing seen yet): the factor multiplies zeros
            const float g = st.m[r] == mx[r] ? 1.f : ex2_approx((st.m[r] - mx[r]) * sc);
            st.m[r] = mx[r];
            st.l[r] *= g;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) { st.o[i][2 * r] *= g; st.o[i][2 * r + 1] *= g; }
        }
    }
    const float b[2] = {mx[0] == kNegInf ? 0.f : mx[0] * sc, mx[1] == kNegInf ? 0.f : mx[1] * sc};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[t][e] = ex2_approx(fmaf(s[t][e], sc, -b[e >> 1]));
            st.l[e >> 1] += s[t][e];
        }
    const uint32_t p0 = pack_bf16x2(s[0][0], s[0][1]), p1 = pack_bf16x2(s[0][2], s[0][3]);
    const uint32_t p2 = pack_bf16x2(s[1][0], s[1][1]), p3 = pack_bf16x2(s[1][2], s[1][3]);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        const uint32_t* v0 = &f.v[c][0].x;
        const uint32_t* v1 = &f.v[c][1].x;
        const uint32_t* v2 = &f.v[c][2].x;
        const uint32_t* v3 = &f.v[c][3].x;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t sel = (e & 1) ? 0x7632 : 0x5410;
            mma_bf16_16816(st.o[c * 8 + e], p0, p1, p2, p3, prmt(v0[e >> 1], v1[e >> 1], sel),
                           prmt(v2[e >> 1], v3[e >> 1], sel), st.o[c * 8 + e]);
        }
    }
}

}  // namespace w4
