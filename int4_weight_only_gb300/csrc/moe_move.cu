// moe_move.cu - tokens copied to their experts' rows, and the experts' rows weighted and
// summed back to tokens.
//
//   out[row[t, j]] = x[t];   out[t] = sum_j w[t, j] y[row[t, j]] (+ shared[t])
//
// Both are bound by HBM: a token's row once on one side, k rows on the other.  A thread takes
// one word of a token's row (16 bytes where rows allow it, else 8 or 4) and all its k
// counterparts, eight at a time, so that their loads or stores are in flight together.  Measured
// in a graph: 8192 tokens of 2048 values to 8 rows each (302 MB) 45.1 us, back 43.3: 0.98 and 1.02
// of the measured copy rate (one row after the other, back: 53); 333 x 3580, 6 rows and a
// shared one (8-byte words) 4.4 us; 16 x 2048 1.7.  2048 tokens of 4096, 4092, 4094 and 4095
// values to 8 rows: 24.4, 27.2, 31.6, 31.2 us there, 21.1, 23.2, 23.7, 41.3 back, with a shared row
// 22.6, 24.7, 25.2, 47.0 (a value a thread: 43 there and 63 back for the last two widths).
#include "block_device.cuh"
#include "w4_internal.h"

#include <algorithm>

namespace w4 {
namespace {

template <int N> struct Word;
template <> struct Word<8> { using T = uint4; };
template <> struct Word<4> { using T = uint2; };
template <> struct Word<2> { using T = uint32_t; };
// Words a thread takes, a CTA's width apart: looking up rows and weights costs as much as a few short words.
template <int N> __host__ __device__ constexpr int words_of() { return N >= 4 ? 1 : 4; }

// ---- rows of any alignment (an odd width): a thread takes 16 bytes of an output row that are
// aligned there, from the two aligned 16-byte words of an input row that hold them.  Elements so near
// the row's ends that those could lie outside it are one a thread.
struct Pieces {
    int head, n, all;                   // elements before, pieces, pieces and single elements

    __device__ __forceinline__ Pieces(const uint16_t* row, int K) {
        head = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 2;
        if (head < 7) head += 8;
        head = min(head, K);
        n = K - head >= 16 ? (K - head - 16) / 8 + 1 : 0;
        all = n + K - 8 * n;
    }
    // the element of single number i >= n
    __device__ __forceinline__ int single(int i) const { return i - n < head ? i - n : i + 7 * n; }
};
struct Eight {
    uint4 a, b;
    int bytes;                          // where the eight start in a, b

    // elements e .. e + 7 of a row; 7 <= e, and e + 16 lies in it
    __device__ __forceinline__ void load(const uint16_t* row, int e) {
        bytes = (int)(reinterpret_cast<uintptr_t>(row + e) & 15);
        const uint4* p = reinterpret_cast<const uint4*>(row + e - bytes / 2);
        a = p[0];
        b = p[1];
    }
    __device__ __forceinline__ uint4 get() const {
        const uint32_t z[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t t[6], u[5];
#pragma unroll
        for (int i = 0; i < 6; ++i) t[i] = bytes & 8 ? z[i + 2] : z[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = bytes & 4 ? t[i + 1] : t[i];
        const int half = (bytes & 2) * 8;
        return make_uint4(__funnelshift_r(u[0], u[1], half), __funnelshift_r(u[1], u[2], half),
                          __funnelshift_r(u[2], u[3], half), __funnelshift_r(u[3], u[4], half));
    }
};

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
    constexpr int W = words_of<N>();
    pdl_wait();
    pdl_launch();
    const int words = a.K / N, c = blockIdx.y * (W * blockDim.x) + threadIdx.x;
    if (c >= words) return;
    const long long t = blockIdx.x;
    const T* x = reinterpret_cast<const T*>(a.x + t * a.stride);
    T v[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        v[i] = T{};
        if (i == 0 || c + i * (int)blockDim.x < words) v[i] = x[c + i * blockDim.x];
    }
    for (int j0 = 0; j0 < a.k; j0 += kRows) {
        int r[kRows];
        rows_of(a, t, j0, c == 0, r);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            if (r[j] < 0) continue;
            T* to = reinterpret_cast<T*>(a.out + (size_t)r[j] * a.K) + c;
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (i == 0 || c + i * (int)blockDim.x < words) to[i * blockDim.x] = v[i];
        }
    }
}

template <int N> __device__ __forceinline__ void add_word(float* acc, typename Word<N>::T u, float w) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const uint32_t z = reinterpret_cast<const uint32_t*>(&u)[i];
        acc[2 * i] = fmaf(w, bf16x2_lo(z), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w, bf16x2_hi(z), acc[2 * i + 1]);
    }
}

template <int N>
__global__ void __launch_bounds__(256) k_moe_combine(const MoveArgs a) {
    using T = typename Word<N>::T;
    constexpr int W = words_of<N>();
    pdl_wait();
    pdl_launch();
    const int words = a.K / N, c = blockIdx.y * (W * blockDim.x) + threadIdx.x;
    if (c >= words) return;
    const long long t = blockIdx.x;
    auto has = [&](int i) { return i == 0 || c + i * (int)blockDim.x < words; };
    float acc[W][N];
    T own[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int e = 0; e < N; ++e) acc[i][e] = 0.f;
        own[i] = T{};
        if (a.shared && has(i)) own[i] = reinterpret_cast<const T*>(a.shared + (size_t)t * a.K)[c + i * blockDim.x];
    }
    for (int j0 = 0; j0 < a.k; j0 += kRows) {
        int r[kRows];
        T u[kRows][W];
        float w[kRows];
        rows_of(a, t, j0, c == 0, r);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            w[j] = r[j] >= 0 ? __ldg(a.weights + t * a.k + j0 + j) : 0.f;
            const T* y = reinterpret_cast<const T*>(a.x + (size_t)max(r[j], 0) * a.K) + c;
#pragma unroll
            for (int i = 0; i < W; ++i) u[j][i] = r[j] >= 0 && has(i) ? __ldcs(y + i * blockDim.x) : T{};
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (r[j] >= 0)
#pragma unroll
                for (int i = 0; i < W; ++i) add_word<N>(acc[i], u[j][i], w[j]);
    }
    T* out = reinterpret_cast<T*>(a.out + (size_t)t * a.K) + c;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if (!has(i)) continue;
        if (a.shared) add_word<N>(acc[i], own[i], 1.f);
        T u;
#pragma unroll
        for (int e = 0; e < N / 2; ++e)
            reinterpret_cast<uint32_t*>(&u)[e] = pack_bf16x2(acc[i][2 * e], acc[i][2 * e + 1]);
        out[i * blockDim.x] = u;
    }
}

__global__ void __launch_bounds__(256) k_moe_gather_any(const MoveArgs a) {
    pdl_wait();
    pdl_launch();
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    const long long t = blockIdx.x;
    const uint16_t* x = a.x + t * a.stride;
    for (int j0 = 0; j0 < a.k; j0 += kRows) {
        int r[kRows];
        rows_of(a, t, j0, c == 0, r);
#pragma unroll 4
        for (int j = 0; j < kRows; ++j) {
            if (r[j] < 0) continue;
            uint16_t* out = a.out + (size_t)r[j] * a.K;
            const Pieces s(out, a.K);
            if (c < s.n) {
                Eight v;
                v.load(x, s.head + 8 * c);
                *reinterpret_cast<uint4*>(out + s.head + 8 * c) = v.get();
            } else if (c < s.all) {
                out[s.single(c)] = x[s.single(c)];
            }
        }
    }
}

__global__ void __launch_bounds__(256) k_moe_combine_any(const MoveArgs a) {
    constexpr int R = 4;                // rows whose loads are in flight together
    pdl_wait();
    pdl_launch();
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    const long long t = blockIdx.x;
    const size_t at = (size_t)t * a.K;
    const Pieces s(a.out + at, a.K);
    if (c >= s.all) return;
    const bool piece = c < s.n;
    const int e = piece ? s.head + 8 * c : s.single(c);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += kRows) {
        int r[kRows];
        rows_of(a, t, j0, c == 0, r);
        auto row = [&](int j) { return a.x + (size_t)r[j] * a.K; };
        auto weight = [&](int j) { return __ldg(a.weights + t * a.k + j0 + j); };
        if (piece) {
#pragma unroll
            for (int j1 = 0; j1 < kRows; j1 += R) {
                Eight v[R];
                float w[R];
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (r[j1 + j] >= 0) {
                        w[j] = weight(j1 + j);
                        v[j].load(row(j1 + j), e);
                    }
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (r[j1 + j] >= 0) add_word<8>(acc, v[j].get(), w[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kRows; ++j)
                if (r[j] >= 0) acc[0] = fmaf(weight(j), bf16_bits_to_f32(row(j)[e]), acc[0]);
        }
    }
    const uint16_t* own = a.shared ? a.shared + at : nullptr;
    uint16_t* out = a.out + at + e;
    if (piece) {
        if (own) {
            Eight v;
            v.load(own, e);
            add_word<8>(acc, v.get(), 1.f);
        }
        *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                                    pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
    } else {
        *out = f32_to_bf16_bits(acc[0] + (own ? bf16_bits_to_f32(own[e]) : 0.f));
    }
}

// `each`: threads that a token needs.
int launch(void (*kern)(const MoveArgs), const MoveArgs& a, int each, cudaStream_t stream) {
    const int threads = std::min(256, (each + 31) / 32 * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T, (unsigned)((each + threads - 1) / threads));
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

template <int N> int threads_of(int K) { return (K / N + words_of<N>() - 1) / words_of<N>(); }
// pieces, and 14 + 23 single elements at most
int threads_of_any(int K) { return K / 8 + std::min(K, 37); }

}  // namespace

int launch_moe_gather(const MoveArgs& a, cudaStream_t stream) {
    switch (row_align(a)) {
        case 16: return launch(k_moe_gather<8>, a, threads_of<8>(a.K), stream);
        case 8: return launch(k_moe_gather<4>, a, threads_of<4>(a.K), stream);
        case 4: return launch(k_moe_gather<2>, a, threads_of<2>(a.K), stream);
        default: return launch(k_moe_gather_any, a, threads_of_any(a.K), stream);
    }
}

int launch_moe_combine(const MoveArgs& a, cudaStream_t stream) {
    switch (row_align(a)) {
        case 16: return launch(k_moe_combine<8>, a, threads_of<8>(a.K), stream);
        case 8: return launch(k_moe_combine<4>, a, threads_of<4>(a.K), stream);
        case 4: return launch(k_moe_combine<2>, a, threads_of<2>(a.K), stream);
        default: return launch(k_moe_combine_any, a, threads_of_any(a.K), stream);
    }
}

}  // namespace w4
