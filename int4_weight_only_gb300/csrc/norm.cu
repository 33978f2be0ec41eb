// norm.cu - the RMS norms after and before a block, with the block's gate,
// residual scale and residual sum, in one pass over the rows.
//
//   u  = y rsqrt(mean(y^2) + eps) (o + w_post)
//   r' = r + a gate u
//   x  = r' rsqrt(mean(r'^2) + eps) (o + w_pre)
//
// A row is read once and kept in registers (EPT elements per thread, V at a
// time) across the two row sums, so HBM sees 8 bytes per element and nothing
// else; everything a row needs is loaded before its first sum, so that a row
// waits for memory once.  Sums and norms are fp32.  Bound by HBM: 8192 rows of
// 3840 take 38.0 us without the norm after the block (0.98 of the measured copy
// rate) and 42.9 us with it (a second row sum), one row 1.7 us of latency.  Rows of
// more than 16384 columns take 1024 threads of 64 registers, which do not hold a
// row's loads (168 bytes spilled): 2048 rows of 16384 take 47.6 / 57.0 us (0.83 /
// 0.69), 1024 of 32768 57.1 / 68.4 (0.69 / 0.58).
#include "block_device.cuh"
#include "w4_internal.h"

#include <algorithm>

namespace w4 {
namespace {

// Sum over the CTA; `red` holds one float per warp and is free again after
// the next __syncthreads.
__device__ __forceinline__ float cta_sum(float v, float* red) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    v = warp_sum(v);
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? red[lane] : 0.f);
}

// V bf16 values as loaded.
template <int V> struct Raw;
template <> struct Raw<8> { uint4 v; };
template <> struct Raw<4> { uint2 v; };
template <> struct Raw<1> { uint16_t v; };

template <int V>
__device__ __forceinline__ Raw<V> load_raw(const uint16_t* p) {
    Raw<V> r;
    if constexpr (V == 8) r.v = *reinterpret_cast<const uint4*>(p);
    else if constexpr (V == 4) r.v = *reinterpret_cast<const uint2*>(p);
    else r.v = *p;
    return r;
}
// Value j of them in fp32.
template <int V>
__device__ __forceinline__ float value(const Raw<V>& r, int j) {
    const uint32_t w = (&r.v.x)[j >> 1];
    return (j & 1) ? bf16x2_hi(w) : bf16x2_lo(w);
}

template <int V>
__device__ __forceinline__ void store_vec(uint16_t* p, const float* f) {
    if constexpr (V == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    } else {
        *p = f32_to_bf16_bits(f[0]);
    }
}

template <int V, int EPT, int MAXT>
__global__ void __launch_bounds__(MAXT, V == 1 ? 1 : EPT == 8 ? 4 : EPT == 16 ? 2 : 1) k_block_norm(const NormArgs a) {
    constexpr int NV = EPT / V;
    __shared__ float red[2][32];
    auto col = [&](int i) { return (i * (int)blockDim.x + (int)threadIdx.x) * V; };
    pdl_wait();
    pdl_launch();
    const int m = blockIdx.x;
    const size_t row = (size_t)m * a.K;
    const float inv_k = 1.f / (float)a.K;
    const uint16_t* grow = a.gate ? a.gate + (size_t)(m / a.gate_div) * a.K : nullptr;
    Raw<V> rr[NV], ry[NV], rg[NV], wo[NV], wi[NV];
    // columns past the row's end repeat its last ones; their values are not used
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = min(col(i), a.K - V);
        if constexpr (V == 1) continue;     // single values would take a register each
        rr[i] = load_raw<V>(a.r + row + c);
        if (a.y) ry[i] = load_raw<V>(a.y + row + c);
        if (grow) rg[i] = load_raw<V>(grow + c);
        if (a.w_post) wo[i] = load_raw<V>(a.w_post + c);
        if (a.x_out) wi[i] = load_raw<V>(a.w_pre + c);
    }
    auto at = [&](const Raw<V>* raw, const uint16_t* p, int i, int j) {
        if constexpr (V == 1) return bf16_bits_to_f32(p[min(col(i), a.K - 1)]);
        else return value<V>(raw[i], j);
    };
    float h[EPT];
    if (a.y) {
        float rs = 1.f;
        if (a.w_post) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float v = col(i) < a.K ? at(ry, a.y + row, i, j) : 0.f;
                    s = fmaf(v, v, s);
                }
            rs = rsqrtf(cta_sum(s, red[0]) * inv_k + a.eps);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float v = at(ry, a.y + row, i, j);
                if (a.w_post) v *= rs * (at(wo, a.w_post, i, j) + a.w_off);
                if (grow) v *= at(rg, grow, i, j);
                h[i * V + j] = fmaf(a.res_scale, v, at(rr, a.r + row, i, j));
            }
            if (col(i) < a.K) store_vec<V>(a.r_out + row + col(i), h + i * V);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) h[i * V + j] = at(rr, a.r + row, i, j);
    }
    if (a.x_out) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float v = col(i) < a.K ? h[i * V + j] : 0.f;
                s = fmaf(v, v, s);
            }
        const float rs = rsqrtf(cta_sum(s, red[1]) * inv_k + a.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (col(i) >= a.K) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) h[i * V + j] *= rs * (at(wi, a.w_pre, i, j) + a.w_off);
            store_vec<V>(a.x_out + row + col(i), h + i * V);
        }
    }
}

template <int V>
int go(const NormArgs& a, cudaStream_t stream) {
    // Elements per thread: 8 in up to 256 threads, then 16 in up to 512 (8192 rows
    // of 3840 with both norms: 42.9 us against 45.1 with 8 in 480 threads and 47.1
    // with 32 in 120); odd rows go by single values, where 8 per thread stay ahead
    // (3841 columns: 112 against 204 us).
    const int ept = a.K <= (V == 1 ? 512 : 256) * 8 ? 8 : a.K <= 512 * 16 ? 16 : 32;
    const int threads = ((a.K + ept - 1) / ept + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.M);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kern = ept == 8 ? k_block_norm<V, 8, 512> : ept == 16 ? k_block_norm<V, 16, 512>
              : threads <= 512 ? k_block_norm<V, 32, 512> : k_block_norm<V, 32, 1024>;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    return e == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

}  // namespace

int launch_block_norm(const NormArgs& a, cudaStream_t stream) {
    // widest vector that every row start and pointer allows
    uintptr_t bits = (uintptr_t)((size_t)a.K * 2);
    for (const void* p : {(const void*)a.y, (const void*)a.r, (const void*)a.w_post, (const void*)a.gate,
                          (const void*)a.w_pre, (const void*)a.r_out, (const void*)a.x_out})
        bits |= (uintptr_t)p;
    if (bits % 16 == 0) return go<8>(a, stream);
    if (bits % 8 == 0) return go<4>(a, stream);
    return go<1>(a, stream);
}

}  // namespace w4
