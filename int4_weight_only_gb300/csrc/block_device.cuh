// block_device.cuh - device helpers of the decoder-block kernels (norms,
// rotary positions, paged attention): programmatic launch, reductions, and
// the cache's addressing with its bounds checks.
#pragma once

#include "w4_device.cuh"

namespace w4 {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float bf16x2_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16x2_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The length of sequence b, clamped to what the table and the launch cover.
__device__ __forceinline__ int kv_length(const w4_paged_kv& kv, int b, int max_len, int* err) {
    const int n = __ldg(kv.kv_len + b);
    const long long cap = min((long long)kv.max_pages * kv.page_size, (long long)max_len);
    const int c = (int)min(max((long long)n, 0LL), cap);
    if (c != n) atomicCAS(err, 0, W4_ERR_PAGE_TABLE);
    return c;
}

// Page number j of sequence b: an entry outside [0, pages) reads as page 0.
__device__ __forceinline__ int page_of(const w4_paged_kv& kv, int b, int j, int* err) {
    const int p = __ldg(kv.table + (long long)b * kv.table_stride + j);
    if ((unsigned)p >= (unsigned)kv.pages) {
        atomicCAS(err, 0, W4_ERR_PAGE_TABLE);
        return 0;
    }
    return p;
}

}  // namespace w4
