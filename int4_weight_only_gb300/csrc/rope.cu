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
// a bf16 rounding.
//
// A CTA takes a token: its threads load their pieces of q, k and v, and meanwhile
// one warp finds the token's sequence and cache slot and computes the
// rot_dim / 2 cosines and sines, in shared memory, for all heads.  Bound by HBM:
// 8152 tokens of 28 + 4 + 4 heads of 128 take 28.8 us (0.77 of the measured copy
// rate; 22.9 us where the slot needs no lookup), one token 3 us of latency.  The
// check of the offsets is in the lookup's own loop: in a warp or a CTA of its own it
// cost 1138 tokens in 24 sequences 1 us of 8.4.
#include "block_device.cuh"
#include "w4_internal.h"

#include <algorithm>

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

// Found by a whole warp: offsets and lengths of 32 sequences in one round of
// loads, then the table's entry.
__device__ __forceinline__ RowPlace place_of(const RopeArgs& a, int t) {
    RowPlace w{0, -1, 0, -1, 0};
    const int lane = threadIdx.x & 31;
    const int cap = (int)min((long long)a.kv.max_pages * a.kv.page_size, (long long)0x7fffffff);
    const int pos = a.pos ? __ldg(a.pos + t) : 0;
    int b = t, ahead = 0, n = 0;                          // ahead: rows of the sequence after t
    if (a.goff) {
        // the last sequence that starts at or before t: offsets do not decrease
        bool found = false;
        int o0 = 0, o1 = 0;
        for (int b0 = 0; b0 < a.kv.batch; b0 += 32) {
            const int i = min(b0 + lane, a.kv.batch - 1);
            const int s0 = __ldg(a.goff + i), s1 = __ldg(a.goff + i + 1), len = __ldg(a.kv.kv_len + i);
            // whether or not a row belongs to the sequence
            if (s0 < 0 || s1 < s0 || s1 > a.T) atomicCAS(a.err, 0, W4_ERR_GROUP_TOKENS);
            const uint32_t m = __ballot_sync(0xffffffffu, b0 + lane < a.kv.batch && s0 <= t);
            if (m) {
                const int f = 31 - __clz(m);
                found = true;
                b = b0 + f;
                o0 = __shfl_sync(0xffffffffu, s0, f);
                o1 = __shfl_sync(0xffffffffu, s1, f);
                n = __shfl_sync(0xffffffffu, len, f);
            }
            if (!(m >> 31) && t < a.T - 1) break;         // the last row sees all offsets
        }
        if (!found || o0 < 0 || o1 > a.T || t >= o1) return w;
        ahead = o1 - 1 - t;
    } else {
        n = __ldg(a.kv.kv_len + b);
    }
    w.have = 1;
    if (n < 0 || n > cap) {
        atomicCAS(a.err, 0, W4_ERR_PAGE_TABLE);
        n = min(max(n, 0), cap);
    }
    w.p = n - 1 - ahead;
    w.P = a.pos ? pos : w.p;
    if (w.p >= 0) {
        const int lg = 31 - __clz(a.kv.page_size);
        const int p = __ldg(a.kv.table + (long long)b * a.kv.table_stride + (w.p >> lg));
        w.slot = w.p & (a.kv.page_size - 1);
        if ((unsigned)p < (unsigned)a.kv.pages) w.page = p;
        else atomicCAS(a.err, 0, W4_ERR_PAGE_TABLE);      // nothing is written
    }
    return w;
}

// VEC: every row start is 16-byte aligned, and chunks of eight never straddle
// the end of the rotated part or of its halves.
template <bool VEC>
__global__ void __launch_bounds__(256, 8) k_rope_append(const RopeArgs a) {
    __shared__ float2 cs[kMaxD / 2];
    __shared__ RowPlace place;
    pdl_wait();
    pdl_launch();
    const int t = blockIdx.x, D = a.kv.head_dim, half = a.rot >> 1;
    const int Hk = a.kv.heads, heads = a.Hq + 2 * Hk;
    auto src_of = [&](int h) {
        return h < a.Hq ? a.q + t * a.q_tok + h * a.q_head
             : h < a.Hq + Hk ? a.k + t * a.k_tok + (h - a.Hq) * a.k_head
                             : a.v + t * a.v_tok + (h - a.Hq - Hk) * a.v_head;
    };
    // VEC pieces of a token: a q or k head has `uq` (in the half layout a piece of
    // the first half and its partner are one), a v head D / 8
    const int uq = a.inter ? D / 8 : (D - half) / 8, uv = D / 8;
    const int total = VEC ? (a.Hq + Hk) * uq + Hk * uv : 0;
    struct Piece { int h, c; bool rot, pair; };
    auto piece = [&](int u) {
        Piece p;
        const int qk = (a.Hq + Hk) * uq;
        if (u < qk) {
            p.h = u / uq;
            p.c = (u - p.h * uq) * 8;
            p.rot = a.inter ? p.c < a.rot : p.c < half;
            p.pair = p.rot && !a.inter;
            if (!a.inter && p.c >= half) p.c += half;     // behind the rotated part
        } else {
            p.h = (u - qk) / uv;
            p.c = (u - qk - p.h * uv) * 8;
            p.h += a.Hq + Hk;
            p.rot = p.pair = false;
        }
        return p;
    };
    uint4 x, y;                                           // a piece, and its partner's
    auto load = [&](int u) {
        if (u >= total) return;
        const Piece p = piece(u);
        const uint16_t* src = src_of(p.h) + p.c;
        x = *reinterpret_cast<const uint4*>(src);
        if (p.pair) y = *reinterpret_cast<const uint4*>(src + half);
    };
    if constexpr (VEC) load(threadIdx.x);
    if (threadIdx.x < 32) {
        const RowPlace p = place_of(a, t);
        if (threadIdx.x == 0) place = p;
        if (p.have)
            for (int i = threadIdx.x; i < half; i += 32) {
                const float2 v = rope_cos_sin(p.P, __ldg(a.inv_freq + i));
                cs[i] = make_float2(v.x * a.mscale, v.y * a.mscale);
            }
    }
    __syncthreads();
    const RowPlace w = place;
    if (!w.have) return;
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
        for (int u = threadIdx.x; u < total; u += blockDim.x) {
            if (u != (int)threadIdx.x) load(u);
            const Piece p = piece(u);
            uint16_t* dst = dst_of(p.h);
            if (!dst) continue;
            dst += p.c;
            uint32_t *xw = &x.x, *yw = &y.x;
            if (none) {
                x = y = make_uint4(0, 0, 0, 0);
            } else if (p.pair) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v0 = cs[p.c + 2 * j], v1 = cs[p.c + 2 * j + 1];
                    const float x0 = bf16x2_lo(xw[j]), x1 = bf16x2_hi(xw[j]);
                    const float y0 = bf16x2_lo(yw[j]), y1 = bf16x2_hi(yw[j]);
                    xw[j] = pack_bf16x2(x0 * v0.x - y0 * v0.y, x1 * v1.x - y1 * v1.y);
                    yw[j] = pack_bf16x2(x0 * v0.y + y0 * v0.x, x1 * v1.y + y1 * v1.x);
                }
            } else if (p.rot) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = cs[(p.c >> 1) + j];
                    const float x0 = bf16x2_lo(xw[j]), y0 = bf16x2_hi(xw[j]);
                    xw[j] = pack_bf16x2(x0 * v.x - y0 * v.y, x0 * v.y + y0 * v.x);
                }
            }
            *reinterpret_cast<uint4*>(dst) = x;
            if (p.pair) *reinterpret_cast<uint4*>(dst + half) = y;
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
            const float p = bf16_bits_to_f32(src[d]), q = bf16_bits_to_f32(src[d2]);
            dst[d] = none ? (uint16_t)0 : f32_to_bf16_bits(p * v.x - q * v.y);
            dst[d2] = none ? (uint16_t)0 : f32_to_bf16_bits(p * v.y + q * v.x);
        }
    }
}

}  // namespace

int launch_rope_append(const RopeArgs& a, cudaStream_t stream) {
    const uintptr_t bits = (uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q_out |
                           (uintptr_t)(2 * (a.q_tok | a.q_head | a.k_tok | a.k_head | a.v_tok | a.v_head));
    const int D = a.kv.head_dim;
    const bool vec = bits % 16 == 0 && a.rot % (a.inter ? 8 : 16) == 0;
    // Two pieces per thread (a piece's loads are one or two 16-byte words): small CTAs
    // and 32 registers keep 2048 threads on an SM, so that a thousand tokens are one wave.
    const int pieces = (a.Hq + a.kv.heads) * (a.inter ? D : D - a.rot / 2) / 8 + a.kv.heads * D / 8;
    const int threads = vec ? std::min(std::max((pieces + 63) / 64 * 32, 64), 256) : 256;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T);
    cfg.blockDim = dim3((unsigned)threads);
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
