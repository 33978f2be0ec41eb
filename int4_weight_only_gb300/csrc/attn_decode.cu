// attn_decode.cu - attention of one new token over the paged cache.
//
//   o = sum_j w_j v_j,  w = softmax over the visible j of scale (q . k_j)
//
// The call is bound by reading the visible keys and values once (4 D bytes a
// key and key-value head); the query heads of a group share that read as the
// rows of one 16-row mma.sync operand (q_heads / heads > 16: several items).
//
// Work: an item is (sequence, key-value head, group of 16 query heads), a unit
// of it 64 keys.  The units of all items form one list, cut into equal
// consecutive shares, one per CTA (two CTAs per SM), so ragged lengths balance
// without the host knowing them.  An item that spans CTAs is joined from fp32
// partial sums by the last of them to arrive, in the list's order: the same
// inputs give the same bits.
//
// A CTA's four warps take 16-key blocks in turn, each with its own online
// softmax.  A lane copies exactly the 16-byte pieces that it will use as
// matrix operands (attn_device.cuh) with cp.async into a private ring in
// shared memory, kStages blocks deep: no barrier inside the loop, and enough
// bytes in flight per SM to cover the latency of HBM.  Keys that the token
// does not see are not read; their pieces are filled with zeros.
#include "attn_device.cuh"
#include "w4_internal.h"

#include <algorithm>

namespace w4 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;
constexpr int kUnitBlocks = kWarps;     // 16-key blocks per unit
constexpr int kRows = 16;               // query heads per item

template <int D> __host__ __device__ constexpr int stage_vecs() { return D / 32 * 2 + D / 64 * 4; }   // per lane
template <int D> __host__ __device__ constexpr int ring_bytes() { return kWarps * kStages * stage_vecs<D>() * 32 * 16; }
// a partial result: o [kRows][D], then m [kRows], l [kRows]
template <int D> __host__ __device__ constexpr int slot_floats() { return kRows * D + 2 * kRows; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
    const int n = read ? 16 : 0;      // 0: fill with zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

struct SeqWork {
    int len;                // clamped length
    KeyBlocks kb;           // its visible 16-key blocks
    int units;              // per item
};

__device__ __forceinline__ SeqWork seq_work(const AttnArgs& a, int b) {
    SeqWork w;
    w.len = kv_length(a.kv, b, a.max_len, a.err);
    w.kb = key_blocks<16>(w.len - 1, w.len - 1, a.window, a.sinks);
    w.units = max(1, (w.kb.n + kUnitBlocks - 1) / kUnitBlocks);   // 0 keys: the unit writes o = 0
    return w;
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_attn_decode(const AttnArgs a) {
    constexpr int SV = stage_vecs<D>();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ long long s_scan[kWarps];
    __shared__ long long s_start;           // first unit of the sequence the share starts in
    __shared__ int s_b, s_last;
    __shared__ float s_ml[kWarps][2][kRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hkv = a.kv.heads, g = a.Hq / Hkv, ngrp = (g + kRows - 1) / kRows;
    const int items = Hkv * ngrp;           // per sequence
    const int B = a.kv.batch;
    pdl_wait();
    pdl_launch();

    // ---- this CTA's share of the unit list
    auto cta_scan = [&](long long v, long long* total) {     // inclusive prefix sum over the CTA
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        __syncthreads();
        if (lane == 31) s_scan[warp] = v;
        __syncthreads();
        long long before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += s_scan[w];
            all += s_scan[w];
        }
        *total = all;
        return v + before;
    };
    auto units_of = [&](int b) { return b < B ? (long long)seq_work(a, b).units * items : 0LL; };
    long long total = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        long long t;
        cta_scan(units_of(b0 + tid), &t);
        total += t;
    }
    const long long share = (total + gridDim.x - 1) / gridDim.x;
    const long long u0 = share * blockIdx.x, u1 = min(u0 + share, total);
    if (u0 >= total) return;
    long long run = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        long long t;
        const long long n = units_of(b0 + tid), incl = run + cta_scan(n, &t);
        if (n > 0 && incl > u0 && incl - n <= u0) { s_b = b0 + tid; s_start = incl - n; }
        run += t;
        if (run > u0) break;
    }
    __syncthreads();
    int b = s_b;
    long long base = s_start;

    uint4* ring = reinterpret_cast<uint4*>(smem) + warp * kStages * SV * 32 + lane;
    const uint32_t ring_s = smem_u32(ring);
    const int lg = 31 - __clz(a.kv.page_size);
    const int ki = lane & 3, kj = lane >> 2;

    for (long long u = u0; u < u1;) {
        const SeqWork w = seq_work(a, b);
        const int it = (int)((u - base) / w.units);
        const long long first_unit = base + (long long)it * w.units;
        const int seg0 = (int)(u - first_unit);
        const int seg1 = (int)(min(u1, first_unit + w.units) - first_unit);
        const int hk = it / ngrp, h0 = hk * g + (it - hk * ngrp) * kRows;
        const int rows = min(kRows, (hk + 1) * g - h0);
        const int p = w.len - 1;

        // ---- query pieces of the lane's two rows
        uint4 qf[D / 32][2];
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                qf[c][r] = kj + 8 * r < rows
                    ? __ldg(reinterpret_cast<const uint4*>(a.q + b * a.q_tok + (h0 + kj + 8 * r) * a.q_head +
                                                           c * 32 + ki * 8))
                    : make_uint4(0, 0, 0, 0);

        // ---- this warp's blocks of the segment: c0, c0 + kWarps, ... below c1
        const int c0 = seg0 * kUnitBlocks + warp, c1 = min(seg1 * kUnitBlocks, w.kb.n);
        const int nb = c0 < c1 ? (c1 - c0 + kWarps - 1) / kWarps : 0;
        const uint16_t* kh = a.kv.k + (long long)hk * a.kv.k_head_stride;
        const uint16_t* vh = a.kv.v + (long long)hk * a.kv.v_head_stride;
        auto seen = [&](int j) { return key_visible(j, p, a.window, a.sinks); };
        auto page_at = [&](int i) {
            return i < nb ? page_of(a.kv, b, (w.kb(c0 + i * kWarps) * 16) >> lg, a.err) : 0;
        };
        auto issue = [&](int i, int page) {
            if (i < nb) {
                const int j0 = w.kb(c0 + i * kWarps) * 16, slot = j0 & (a.kv.page_size - 1);
                const uint32_t dst = ring_s + (i % kStages) * SV * 512;
                const uint16_t* kp = kh + page * a.kv.k_page_stride;
                const uint16_t* vp = vh + page * a.kv.v_page_stride;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int key = kj + 8 * t;
                    const bool rd = seen(j0 + key);
                    const uint16_t* src = kp + (slot + key) * a.kv.k_slot_stride + ki * 8;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) cp_async16(dst + (c * 2 + t) * 512, src + c * 32, rd);
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int key = 2 * ki + (n & 1) + 8 * (n >> 1);
                    const bool rd = seen(j0 + key);
                    const uint16_t* src = vp + (slot + key) * a.kv.v_slot_stride + kj * 8;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        cp_async16(dst + (D / 32 * 2 + c * 4 + n) * 512, src + c * 64, rd);
                }
            }
            cp_commit();
        };

        RowState<D> st;
        st.init();
        int pg = page_at(0);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            const int nx = page_at(i + 1);
            issue(i, pg);
            pg = nx;
        }
        for (int i = 0; i < nb; ++i) {
            cp_wait<kStages - 2>();
            const uint4* sp = ring + (i % kStages) * SV * 32;
            Frag<D> f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
#pragma unroll
                for (int t = 0; t < 2; ++t) f.k[c][t] = sp[(c * 2 + t) * 32];
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int n = 0; n < 4; ++n) f.v[c][n] = sp[(D / 32 * 2 + c * 4 + n) * 32];
            // the slot of block i - 1 was read into registers before this point
            const int nx = page_at(i + kStages);
            issue(i + kStages - 1, pg);
            pg = nx;
            const int j0 = w.kb(c0 + i * kWarps) * 16;
            bool vis[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) vis[t][e] = seen(j0 + 8 * t + 2 * ki + (e & 1));
            attn_step<D>(st, qf, f, vis, a.scale);
        }
        cp_wait<0>();

        // ---- join the warps in shared memory (the ring is idle)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
            st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
            if (ki == 0) { s_ml[warp][0][kj + 8 * r] = st.m[r]; s_ml[warp][1][kj + 8 * r] = st.l[r]; }
        }
        __syncthreads();
        float* so = reinterpret_cast<float*>(smem);           // [kWarps][kRows][D]
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                so[(warp * kRows + kj + 8 * (e >> 1)) * D + out_col(nt, e, lane)] = st.o[nt][e];
        __syncthreads();

        const bool whole = seg0 == 0 && seg1 == w.units;
        const int first = (int)(first_unit / share), last = (int)((first_unit + w.units - 1) / share);
        float* slots = a.partial;
        auto slot_of = [&](int cta) { return slots + (size_t)(2 * cta + (cta > first ? 0 : 1)) * slot_floats<D>(); };
        float* mine = slot_of((int)blockIdx.x);
        auto put = [&](int r, int d, float o, float m, float l) {       // a finished row's value
            a.out[((size_t)b * a.Hq + h0 + r) * D + d] = f32_to_bf16_bits(l == 0.f ? 0.f : o / l);
            if (a.lse && d == 0)
                a.lse[(size_t)b * a.Hq + h0 + r] =
                    l == 0.f ? kNegInf : (m * a.scale + log2f(l)) * 0.6931471805599453f;
        };
        for (int i = tid; i < rows * D; i += kThreads) {
            const int r = i / D, d = i - r * D;
            float m = kNegInf, l = 0.f, o = 0.f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) m = fmaxf(m, s_ml[x][0][r]);
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float mw = s_ml[x][0][r];
                const float fac = mw == m ? 1.f : ex2_approx((mw - m) * a.scale);
                l += fac * s_ml[x][1][r];
                o += fac * so[(x * kRows + r) * D + d];
            }
            if (whole) {
                put(r, d, o, m, l);
            } else {
                mine[r * D + d] = o;
                if (d == 0) { mine[kRows * D + r] = m; mine[kRows * D + kRows + r] = l; }
            }
        }
        if (!whole) {
            const int n = last - first + 1;
            __syncthreads();
            if (tid == 0) {
                const bool is_last = atom_add_acq_rel_gpu(a.tickets + first, 1) == n - 1;
                if (is_last) a.tickets[first] = 0;
                s_last = is_last;
            }
            __syncthreads();
            if (s_last) {
                // factors exp2((m_i - m) scale) of the parts, then the sums in part order
                float* fac = reinterpret_cast<float*>(smem);          // [n][kRows]
                for (int r = warp; r < rows; r += kWarps) {
                    float m = kNegInf, l = 0.f;
                    for (int i = lane; i < n; i += 32) m = fmaxf(m, ld_cg(slot_of(first + i) + kRows * D + r));
#pragma unroll
                    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    for (int i = lane; i < n; i += 32) {
                        const float* s = slot_of(first + i) + kRows * D;
                        const float mi = ld_cg(s + r), fi = mi == m ? 1.f : ex2_approx((mi - m) * a.scale);
                        fac[i * kRows + r] = fi;
                        l += fi * ld_cg(s + kRows + r);
                    }
                    l = warp_sum(l);
                    if (lane == 0) { s_ml[0][0][r] = m; s_ml[0][1][r] = l; }
                }
                __syncthreads();
                for (int i = tid; i < rows * D; i += kThreads) {
                    const int r = i / D, d = i - r * D;
                    float o = 0.f;
#pragma unroll 8
                    for (int x = 0; x < n; ++x)
                        o += fac[x * kRows + r] * ld_cg(slot_of(first + x) + r * D + d);
                    put(r, d, o, s_ml[0][0][r], s_ml[0][1][r]);
                }
            }
        }
        __syncthreads();
        u = first_unit + seg1;
        if (u == base + (long long)w.units * items) { base = u; ++b; }
    }
}

template <int D>
int go(const AttnArgs& a, int sm_count, cudaStream_t stream) {
    constexpr int bytes = ring_bytes<D>();
    static_assert(kWarps * kRows * D * 4 <= bytes, "the warps' outputs fit the ring");
    if (cudaFuncSetAttribute(k_attn_decode<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return W4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sm_count * kCtasPerSm));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attn_decode<D>, a) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

}  // namespace

size_t attn_decode_ws_bytes(int, int, int, int D, int sm_count) {
    return (size_t)sm_count * kCtasPerSm * 2 * (kRows * D + 2 * kRows) * sizeof(float);
}

int launch_attn_decode(const AttnArgs& a, int sm_count, cudaStream_t stream) {
    return a.kv.head_dim == 128 ? go<128>(a, sm_count, stream) : go<64>(a, sm_count, stream);
}

}  // namespace w4
