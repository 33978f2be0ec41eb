// attn_prefill.cu - attention of a prompt, or of a chunk behind a cached
// prefix, over the paged cache (the rule of attn_decode.cu for every token).
//
// The rows of a tile are (token, query head of one key-value head), so a
// group's heads share the keys and values they read.  A warp owns 16 rows and
// walks the 16-key blocks that any of them sees.
#include "attn_device.cuh"
#include "w4_internal.h"

#include <algorithm>

namespace w4 {
namespace {

constexpr int kWarps = 4;
constexpr int kTileRows = 16 * kWarps;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) k_attn_prefill(const AttnArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ki = lane & 3, kj = lane >> 2;
    const int b = blockIdx.z, hk = blockIdx.y, g = a.Hq / a.kv.heads;
    pdl_wait();
    pdl_launch();
    int t0, t1;
    seq_rows(a.goff, b, a.T, &t0, &t1, a.err);
    const int nq = t1 - t0;
    if (nq > a.max_q) {
        if (threadIdx.x == 0) atomicCAS(a.err, 0, W4_ERR_GROUP_TOKENS);
        return;
    }
    const int row0 = (blockIdx.x * kWarps + warp) * 16;
    if (row0 >= nq * g) return;
    const int len = kv_length(a.kv, b, a.max_len, a.err);
    const int lg = 31 - __clz(a.kv.page_size);
    // the lane's two rows: token, position, query head
    int tok[2], pos[2], head[2];
    bool have[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = row0 + kj + 8 * r;
        have[r] = row < nq * g;
        tok[r] = t0 + row / g;
        pos[r] = have[r] ? len - nq + row / g : -1;
        head[r] = hk * g + row % g;
    }
    uint4 qf[D / 32][2];
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            qf[c][r] = have[r] ? __ldg(reinterpret_cast<const uint4*>(a.q + tok[r] * a.q_tok + head[r] * a.q_head +
                                                                      c * 32 + ki * 8))
                               : make_uint4(0, 0, 0, 0);
    const int p0 = len - nq + row0 / g, p1 = len - nq + min(row0 + 15, nq * g - 1) / g;
    const KeyBlocks kb = key_blocks<16>(max(p0, 0), p1, a.window, a.sinks);
    const uint16_t* kh = a.kv.k + (long long)hk * a.kv.k_head_stride;
    const uint16_t* vh = a.kv.v + (long long)hk * a.kv.v_head_stride;
    RowState<D> st;
    st.init();
    for (int c = 0; c < kb.n; ++c) {
        const int j0 = kb(c) * 16, slot = j0 & (a.kv.page_size - 1);
        const int page = page_of(a.kv, b, j0 >> lg, a.err);
        Frag<D> f;
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int key = kj + 8 * t;
            const uint16_t* src = kh + page * a.kv.k_page_stride + (slot + key) * a.kv.k_slot_stride + ki * 8;
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
                f.k[x][t] = j0 + key < len ? __ldg(reinterpret_cast<const uint4*>(src + x * 32)) : zero;
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int key = 2 * ki + (n & 1) + 8 * (n >> 1);
            const uint16_t* src = vh + page * a.kv.v_page_stride + (slot + key) * a.kv.v_slot_stride + kj * 8;
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                f.v[x][n] = j0 + key < len ? __ldg(reinterpret_cast<const uint4*>(src + x * 64)) : zero;
        }
        bool vis[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                vis[t][e] = key_visible(j0 + 8 * t + 2 * ki + (e & 1), pos[e >> 1], a.window, a.sinks);
        attn_step<D>(st, qf, f, vis, a.scale);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float l = st.l[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (!have[r]) continue;
        const size_t at = (size_t)tok[r] * a.Hq + head[r];
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float o = st.o[nt][2 * r + e];
                a.out[at * D + out_col(nt, e, lane)] = f32_to_bf16_bits(l == 0.f ? 0.f : o / l);
            }
        if (a.lse && ki == 0)
            a.lse[at] = l == 0.f ? kNegInf : (st.m[r] * a.scale + log2f(l)) * 0.6931471805599453f;
    }
}

}  // namespace

size_t attn_prefill_ws_bytes(int, int, int, int, int, int, int) { return 0; }

int launch_attn_prefill(const AttnArgs& a, int sm_count, cudaStream_t stream) {
    const int g = a.Hq / a.kv.heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)a.max_q * g + kTileRows - 1) / kTileRows),
                       (unsigned)a.kv.heads, (unsigned)a.kv.batch);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = a.kv.head_dim == 128 ? cudaLaunchKernelEx(&cfg, k_attn_prefill<128>, a)
                                               : cudaLaunchKernelEx(&cfg, k_attn_prefill<64>, a);
    return e == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

}  // namespace w4
