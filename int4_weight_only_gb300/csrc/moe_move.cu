// moe_move.cu - tokens copied to their experts' rows, and the experts' rows weighted and
// summed back to tokens.
//
//   out[row[t, j]] = x[t];   out[t] = sum_j w[t, j] y[row[t, j]] (+ shared[t])
//
// Both are bound by HBM: a token's row once on one side, k rows on the other.  A thread takes
// one word of a token's row (16 bytes where rows allow it, else 8 or 2) and all its k
// counterparts, eight at a time, so that their loads or stores are in flight together.  Measured
// in a graph: 8192 tokens of 2048 values to 8 rows each (302 MB) 45.1 us, back 43.3: 0.98 and 1.02
// of the measured copy rate (one row after the other, back: 53); 333 x 3580, 6 rows and a
// shared one (8-byte words) 4.6 us; 16 x 2048 1.6.
#include "block_device.cuh"
#include "w4_internal.h"

#include <algorithm>

namespace w4 {
namespace {

template <int N> struct Word;
template <> struct Word<8> { using T = uint4; };
template <> struct Word<4> { using T = uint2; };
template <> struct Word<1> { using T = uint16_t; };

// Rows j0 .. j0 + 7 of token t, -1 where there is none; `tell` reports the wrong ones.
constexpr int kRows = 8;
__device__ __forceinline__ void rows_of(const MoveArgs& a, long long t, int j0, bool tell, int* r) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) r[j] = j0 + j < a.k ? __ldg(a.row + t * a.k + j0 + j) : -1;
#pragma unroll
    for (int j = 0; j < kRows; ++j)
        if ((unsigned)r[j] >= (unsigned)a.R) {
            if (tell && r[j] != -1) atomicCAS(a.err, 0, W4_ERR_GROUP_TOKENS);
            r[j] = -1;
        }
}

template <int N>
__global__ void __launch_bounds__(256) k_moe_gather(const MoveArgs a) {
    using T = typename Word<N>::T;
    pdl_wait();
    pdl_launch();
    const int words = a.K / N, c = blockIdx.y * blockDim.x + threadIdx.x;
    if (c >= words) return;
    const long long t = blockIdx.x;
    const T v = *reinterpret_cast<const T*>(a.x + t * a.stride + (size_t)c * N);
    for (int j0 = 0; j0 < a.k; j0 += kRows) {
        int r[kRows];
        rows_of(a, t, j0, c == 0, r);
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (r[j] >= 0) *reinterpret_cast<T*>(a.out + (size_t)r[j] * a.K + (size_t)c * N) = v;
    }
}

template <int N> __device__ __forceinline__ void add_word(float* acc, typename Word<N>::T u, float w) {
    if constexpr (N == 1) {
        acc[0] = fmaf(w, bf16_bits_to_f32(u), acc[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint32_t z = (&u.x)[i];
            acc[2 * i] = fmaf(w, bf16x2_lo(z), acc[2 * i]);
            acc[2 * i + 1] = fmaf(w, bf16x2_hi(z), acc[2 * i + 1]);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(256) k_moe_combine(const MoveArgs a) {
    using T = typename Word<N>::T;
    pdl_wait();
    pdl_launch();
    const int words = a.K / N, c = blockIdx.y * blockDim.x + threadIdx.x;
    if (c >= words) return;
    const long long t = blockIdx.x;
    const size_t at = (size_t)t * a.K + (size_t)c * N;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    T own{};
    if (a.shared) own = *reinterpret_cast<const T*>(a.shared + at);
    for (int j0 = 0; j0 < a.k; j0 += kRows) {
        int r[kRows];
        T u[kRows];
        float w[kRows];
        rows_of(a, t, j0, c == 0, r);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            w[j] = r[j] >= 0 ? __ldg(a.weights + t * a.k + j0 + j) : 0.f;
            u[j] = r[j] >= 0 ? __ldcs(reinterpret_cast<const T*>(a.x + (size_t)r[j] * a.K + (size_t)c * N)) : T{};
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (r[j] >= 0) add_word<N>(acc, u[j], w[j]);
    }
    if (a.shared) add_word<N>(acc, own, 1.f);
    if constexpr (N == 1) {
        a.out[at] = f32_to_bf16_bits(acc[0]);
    } else {
        typename Word<N>::T u;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) (&u.x)[i] = pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
        *reinterpret_cast<typename Word<N>::T*>(a.out + at) = u;
    }
}

int launch(void (*kern)(const MoveArgs), const MoveArgs& a, int words, cudaStream_t stream) {
    const int threads = std::min(256, (words + 31) / 32 * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T, (unsigned)((words + threads - 1) / threads));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

// Bytes that every row of the call starts at a multiple of.
int row_align(const MoveArgs& a) {
    const uintptr_t bits = (uintptr_t)a.x | (uintptr_t)a.out | (uintptr_t)a.shared | (uintptr_t)(2 * a.stride) |
                           (uintptr_t)(2 * a.K);
    return (int)std::min<uintptr_t>(bits & ~(bits - 1), 16);
}

}  // namespace

int launch_moe_gather(const MoveArgs& a, cudaStream_t stream) {
    const int n = row_align(a);
    return n == 16 ? launch(k_moe_gather<8>, a, a.K / 8, stream)
         : n == 8 ? launch(k_moe_gather<4>, a, a.K / 4, stream) : launch(k_moe_gather<1>, a, a.K, stream);
}

int launch_moe_combine(const MoveArgs& a, cudaStream_t stream) {
    const int n = row_align(a);
    return n == 16 ? launch(k_moe_combine<8>, a, a.K / 8, stream)
         : n == 8 ? launch(k_moe_combine<4>, a, a.K / 4, stream) : launch(k_moe_combine<1>, a, a.K, stream);
}

}  // namespace w4
