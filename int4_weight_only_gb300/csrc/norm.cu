// norm.cu - the RMS norms after and before a block, with the block's gate,
// residual scale and residual sum, in one pass over the rows.
//
//   u  = y rsqrt(mean(y^2) + eps) (o + w_post)
//   r' = r + a gate u
//   x  = r' rsqrt(mean(r'^2) + eps) (o + w_pre)
//
// A row is read once and kept in registers (EPT elements per thread, V at a
// time) across the two row sums, so HBM sees 8 bytes per element and nothing
// else.  Sums and norms are fp32.
#include "block_device.cuh"
#include "w4_internal.h"

namespace w4 {
namespace {

// Sum over the CTA; `red` holds one float per warp and is free again after
// the next __syncthreads.
__device__ __forceinline__ float cta_sum(float v, float* red) {
    const int warps = blockDim.x >> 5;
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < warps; ++i) t += red[i];
    return t;
}

template <int V>
__device__ __forceinline__ void load_vec(const uint16_t* p, float* f) {
    if constexpr (V == 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        f[0] = bf16x2_lo(w.x); f[1] = bf16x2_hi(w.x); f[2] = bf16x2_lo(w.y); f[3] = bf16x2_hi(w.y);
        f[4] = bf16x2_lo(w.z); f[5] = bf16x2_hi(w.z); f[6] = bf16x2_lo(w.w); f[7] = bf16x2_hi(w.w);
    } else if constexpr (V == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        f[0] = bf16x2_lo(w.x); f[1] = bf16x2_hi(w.x); f[2] = bf16x2_lo(w.y); f[3] = bf16x2_hi(w.y);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = bf16_bits_to_f32(p[i]);
    }
}

template <int V>
__device__ __forceinline__ void store_vec(uint16_t* p, const float* f) {
    if constexpr (V == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = f32_to_bf16_bits(f[i]);
    }
}

template <int V, int EPT>
__global__ void __launch_bounds__(EPT == 32 ? 1024 : 512) k_block_norm(const NormArgs a) {
    constexpr int NV = EPT / V;
    __shared__ float red[2][32];
    pdl_wait();
    pdl_launch();
    const float inv_k = 1.f / (float)a.K;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
        const size_t row = (size_t)m * a.K;
        float h[EPT];
        auto col = [&](int i) { return (i * (int)blockDim.x + (int)threadIdx.x) * V; };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (col(i) < a.K) load_vec<V>((a.y ? a.y : a.r) + row + col(i), h + i * V);
            else for (int j = 0; j < V; ++j) h[i * V + j] = 0.f;
        }
        if (a.y) {
            if (a.w_post) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < EPT; ++i) s = fmaf(h[i], h[i], s);
                const float rs = rsqrtf(cta_sum(s, red[0]) * inv_k + a.eps);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (col(i) >= a.K) continue;
                    float w[V];
                    load_vec<V>(a.w_post + col(i), w);
#pragma unroll
                    for (int j = 0; j < V; ++j) h[i * V + j] *= rs * (w[j] + a.w_off);
                }
            }
            const uint16_t* grow = a.gate ? a.gate + (size_t)(m / a.gate_div) * a.K : nullptr;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (col(i) >= a.K) continue;
                float r[V];
                load_vec<V>(a.r + row + col(i), r);
                if (grow) {
                    float g[V];
                    load_vec<V>(grow + col(i), g);
#pragma unroll
                    for (int j = 0; j < V; ++j) h[i * V + j] *= g[j];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) h[i * V + j] = fmaf(a.res_scale, h[i * V + j], r[j]);
                store_vec<V>(a.r_out + row + col(i), h + i * V);
            }
        }
        if (a.x_out) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < EPT; ++i) s = fmaf(h[i], h[i], s);
            const float rs = rsqrtf(cta_sum(s, red[1]) * inv_k + a.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (col(i) >= a.K) continue;
                float w[V];
                load_vec<V>(a.w_pre + col(i), w);
#pragma unroll
                for (int j = 0; j < V; ++j) h[i * V + j] *= rs * (w[j] + a.w_off);
                store_vec<V>(a.x_out + row + col(i), h + i * V);
            }
        }
        __syncthreads();   // red is written again by the next row
    }
}

template <int V>
int go(const NormArgs& a, int sm_count, cudaStream_t stream) {
    // the fewest elements per thread that keep the CTA at 512 threads
    const int ept = a.K <= 512 * 8 ? 8 : a.K <= 512 * 16 ? 16 : 32;
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
    cudaError_t e = ept == 8 ? cudaLaunchKernelEx(&cfg, k_block_norm<V, 8>, a)
                  : ept == 16 ? cudaLaunchKernelEx(&cfg, k_block_norm<V, 16>, a)
                              : cudaLaunchKernelEx(&cfg, k_block_norm<V, 32>, a);
    return e == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

}  // namespace

int launch_block_norm(const NormArgs& a, int sm_count, cudaStream_t stream) {
    // widest vector that every row start and pointer allows
    uintptr_t bits = (uintptr_t)((size_t)a.K * 2);
    for (const void* p : {(const void*)a.y, (const void*)a.r, (const void*)a.w_post, (const void*)a.gate,
                          (const void*)a.w_pre, (const void*)a.r_out, (const void*)a.x_out})
        bits |= (uintptr_t)p;
    if (bits % 16 == 0) return go<8>(a, sm_count, stream);
    if (bits % 8 == 0) return go<4>(a, sm_count, stream);
    return go<1>(a, sm_count, stream);
}

}  // namespace w4
