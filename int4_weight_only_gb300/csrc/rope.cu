// rope.cu - rotary positions on q and k, and k and v written into the paged
// cache, in one pass over the rows of a qkv projection.
//
//   (a, c) -> mscale (a cos - c sin, a sin + c cos),  angle = P inv_freq[i]
//
// The product of a position and a frequency needs more than 24 bits: at
// position 131071 its fp32 rounding is 0.004 rad.  It is taken as p + e
// (p = fl(P f), e = fma(P, f, -p), exact) and reduced modulo 2 pi in steps
// (Cody and Waite): k = rint(p / 2 pi), r = p - k C1 - k C2 + e with
// C1 + C2 = 2 pi; the first step is exact since p and k C1 are close.  With
// |r| <= pi the fast sine and cosine are good to 2^-21 (absolute), far below
// a bf16 rounding.  A CTA computes a token's rot_dim / 2 pairs once, in shared
// memory, for all its heads.
#include "block_device.cuh"
#include "w4_internal.h"

namespace w4 {
namespace {

constexpr int kMaxD = 256;

__device__ __forceinline__ float2 rope_cos_sin(int P, float f) {
    const float C1 = 6.283185482025146484375f;           // fl(2 pi)
    const float C2 = -1.74845553146951e-7f;              // 2 pi - C1
    const float pf = (float)P;
    const float p = __fmul_rn(pf, f);
    const float e = fmaf(pf, f, -p);
    const float k = rintf(p * 0.15915494309189535f);
    float r = fmaf(-k, C1, p);
    r = fmaf(-k, C2, r) + e;
    return make_float2(__cosf(r), __sinf(r));
}

// Where one row goes: its sequence's cache slot and rotary position.
struct RowPlace {
    int have;          // the row belongs to a sequence
    int p, P;          // token index (negative: none), rotary position
    int page, slot;    // page < 0: not written
};

__device__ RowPlace place_of(const RopeArgs& a, int t) {
    RowPlace w{0, -1, 0, -1, 0};
    int b = t, ahead = 0;                                 // rows of the sequence after t
    if (a.goff) {
        int lo = 0, hi = a.kv.batch;                      // last b with goff[b] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.goff + mid) <= t) lo = mid; else hi = mid;
        }
        b = lo;
        int t0, t1;
        seq_rows(a.goff, b, a.T, &t0, &t1, a.err);
        if (t < t0 || t >= t1) return w;
        ahead = t1 - 1 - t;
    }
    w.have = 1;
    const long long cap = (long long)a.kv.max_pages * a.kv.page_size;
    const int n = kv_length(a.kv, b, (int)min(cap, (long long)0x7fffffff), a.err);
    w.p = n - 1 - ahead;
    w.P = a.pos ? __ldg(a.pos + t) : w.p;
    if (w.p >= 0) {
        const int p = __ldg(a.kv.table + (long long)b * a.kv.table_stride + w.p / a.kv.page_size);
        w.slot = w.p % a.kv.page_size;
        if ((unsigned)p < (unsigned)a.kv.pages) w.page = p;
        else atomicCAS(a.err, 0, W4_ERR_PAGE_TABLE);      // nothing is written
    }
    return w;
}

// VEC: every row start is 16-byte aligned, and chunks of eight never straddle
// the end of the rotated part or of its halves.
template <bool VEC>
__global__ void __launch_bounds__(256) k_rope_append(const RopeArgs a) {
    __shared__ float2 cs[kMaxD / 2];
    __shared__ RowPlace place;
    pdl_wait();
    pdl_launch();
    const int t = blockIdx.x, D = a.kv.head_dim, half = a.rot >> 1;
    if (threadIdx.x == 0) place = place_of(a, t);
    __syncthreads();
    const RowPlace w = place;
    if (!w.have) return;
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
        float2 v = rope_cos_sin(w.P, __ldg(a.inv_freq + i));
        cs[i] = make_float2(v.x * a.mscale, v.y * a.mscale);
    }
    __syncthreads();
    const int Hk = a.kv.heads, heads = a.Hq + 2 * Hk;
    auto src_of = [&](int h) {
        return h < a.Hq ? a.q + t * a.q_tok + h * a.q_head
             : h < a.Hq + Hk ? a.k + t * a.k_tok + (h - a.Hq) * a.k_head
                             : a.v + t * a.v_tok + (h - a.Hq - Hk) * a.v_head;
    };
    auto dst_of = [&](int h) -> uint16_t* {
        if (h < a.Hq) return a.q_out + ((size_t)t * a.Hq + h) * D;
        if (w.page < 0) return nullptr;
        if (h < a.Hq + Hk)
            return a.kv.k + w.page * a.kv.k_page_stride + (h - a.Hq) * a.kv.k_head_stride +
                   w.slot * a.kv.k_slot_stride;
        return a.kv.v + w.page * a.kv.v_page_stride + (h - a.Hq - Hk) * a.kv.v_head_stride +
               w.slot * a.kv.v_slot_stride;
    };
    const bool none = w.p < 0;                            // an unused batch row: q_out = 0
    if constexpr (VEC) {
        const int chunks = D / 8;
        for (int i = threadIdx.x; i < heads * chunks; i += blockDim.x) {
            const int h = i / chunks, c = (i - h * chunks) * 8;
            const bool rot = h < a.Hq + Hk && c < a.rot;
            // half layout: the chunk of first halves also does its partner
            if (rot && !a.inter && c >= half) continue;
            uint16_t* dst = dst_of(h);
            if (!dst) continue;
            const uint16_t* src = src_of(h);
            uint4 u = *reinterpret_cast<const uint4*>(src + c), o;
            if (none) {
                *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
                if (rot && !a.inter) *reinterpret_cast<uint4*>(dst + c + half) = make_uint4(0, 0, 0, 0);
                continue;
            }
            if (!rot) {
                *reinterpret_cast<uint4*>(dst + c) = u;
            } else if (a.inter) {
                uint32_t* uw = &u.x;
                uint32_t* ow = &o.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = cs[(c >> 1) + j];
                    const float x = bf16x2_lo(uw[j]), y = bf16x2_hi(uw[j]);
                    ow[j] = pack_bf16x2(x * v.x - y * v.y, x * v.y + y * v.x);
                }
                *reinterpret_cast<uint4*>(dst + c) = o;
            } else {
                uint4 u2 = *reinterpret_cast<const uint4*>(src + c + half), o2;
                uint32_t *uw = &u.x, *ow = &o.x, *uw2 = &u2.x, *ow2 = &o2.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v0 = cs[c + 2 * j], v1 = cs[c + 2 * j + 1];
                    const float x0 = bf16x2_lo(uw[j]), x1 = bf16x2_hi(uw[j]);
                    const float y0 = bf16x2_lo(uw2[j]), y1 = bf16x2_hi(uw2[j]);
                    ow[j] = pack_bf16x2(x0 * v0.x - y0 * v0.y, x1 * v1.x - y1 * v1.y);
                    ow2[j] = pack_bf16x2(x0 * v0.y + y0 * v0.x, x1 * v1.y + y1 * v1.x);
                }
                *reinterpret_cast<uint4*>(dst + c) = o;
                *reinterpret_cast<uint4*>(dst + c + half) = o2;
            }
        }
    } else {
        for (int i = threadIdx.x; i < heads * D; i += blockDim.x) {
            const int h = i / D, d = i - h * D;
            const bool rot = h < a.Hq + Hk && d < a.rot;
            // a rotated pair is done by its first element
            if (rot && (a.inter ? (d & 1) : d >= half)) continue;
            uint16_t* dst = dst_of(h);
            if (!dst) continue;
            const uint16_t* src = src_of(h);
            const int d2 = a.inter ? d + 1 : d + half;
            if (!rot) {
                dst[d] = none ? (uint16_t)0 : src[d];
                continue;
            }
            const float2 v = cs[a.inter ? d >> 1 : d];
            const float x = bf16_bits_to_f32(src[d]), y = bf16_bits_to_f32(src[d2]);
            dst[d] = none ? (uint16_t)0 : f32_to_bf16_bits(x * v.x - y * v.y);
            dst[d2] = none ? (uint16_t)0 : f32_to_bf16_bits(x * v.y + y * v.x);
        }
    }
}

}  // namespace

int launch_rope_append(const RopeArgs& a, cudaStream_t stream) {
    const uintptr_t bits = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q_out |
                           (uintptr_t)(2 * (a.q_tok | a.q_head | a.k_tok | a.k_head | a.v_tok | a.v_head));
    const bool vec = bits % 16 == 0 && a.rot % (a.inter ? 8 : 16) == 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, k_rope_append<true>, a)
                              : cudaLaunchKernelEx(&cfg, k_rope_append<false>, a);
    return e == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

}  // namespace w4
