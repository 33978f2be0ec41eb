// attn_prefill.cu - attention of a prompt, or of a chunk behind a cached
// prefix, over the paged cache (the rule of attn_decode.cu for every token),
// on the 5th-generation tensor cores.
//
//   S = Q K^T,  P = exp2(c S - c m),  O = P V / sum(P)
//
// A query tile is 128 rows (tokens x query heads of one key-value head, so the
// heads of a group share the keys and values), a step 128 keys.  One CTA per
// SM works on two tiles A and B over the same keys: while the tensor cores
// compute one tile's S and O, the other tile's warps take its exponentials.
//
// TMEM (512 columns): S_A, S_B (128 each), O_A, O_B (D each).  P is written as
// bf16 over the S it came from and is the next product's A operand, straight
// from TMEM; O is accumulated in TMEM over all steps.
//
// The running maximum m is lazy: a row keeps the maximum it scaled by until a
// step exceeds it by more than 2^8, so O is rescaled in the first steps and
// then hardly ever; P stays below 2^8, which costs bf16 nothing.  The sums use
// the fp32 weights, before they are rounded to bf16 as matrix operands.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax of tile A, B: one row per thread
//   warp 8          TMA: Q once, then K and V blocks into a ring of slots (K
//                   in even, V in odd slots), one box per page and 64 columns;
//                   pages past the sequence's end are read out of bounds of
//                   the tensor map, which fills them with zeros
//   warp 9          TMEM allocation; one thread issues the MMAs, for each step
//                   O_A += P_A V, S_A = Q_A K', O_B += P_B V, S_B = Q_B K'
//   warps 10, 11    release V blocks to the MMAs.  In a block that not every
//                   row sees entirely, a weight of zero does not make a NaN
//                   harmless: slots past the end are zeroed, and if a hidden
//                   slot holds a NaN or infinity the tiles are recomputed row
//                   by row at the end (attend_row)
// Every wait is bounded (mbar_wait); copies and MMAs in flight are drained
// before the CTA ends.
#include "attn_device.cuh"
#include "w4_internal.h"

#include <algorithm>
#include <cstring>

namespace w4 {
namespace {

constexpr int kN = 128;                 // keys per step
constexpr int kTile = 128;              // rows per query tile
constexpr int kThreads = 384;
constexpr float kLazy = 8.f;            // log2 units the maximum may lag behind

template <int D> __host__ __device__ constexpr int slots() { return D == 128 ? 4 : 8; }
template <int D> __host__ __device__ constexpr int slot_bytes() { return kN * D * 2; }

struct Ctl {
    uint64_t qfull;
    uint64_t full[8], empty[8], vready[8];
    uint64_t sfull[2], pready[2], ofull[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    int bad;            // a block that some row does not see holds a non-finite value
};

template <int D> __host__ __device__ constexpr size_t smem_total() {
    return 1024 + 2 * kTile * D * 2 + (size_t)slots<D>() * slot_bytes<D>() + sizeof(Ctl);
}

// D[tmem] (+)= A[tmem] * B[smem desc]: the A operand is 128 lanes of bf16
// pairs, 8 columns per 16-wide step.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(acc) : "memory");
}

// Shared-memory descriptor of a B operand stored [k][n] with n contiguous (MN
// major), 128-byte swizzle: 64-column panels of 128-byte rows; panels LBO
// apart, groups of 8 rows (1024 bytes) SBO apart.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t panel_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(panel_bytes >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// 16 TMEM columns of this warp's lanes from registers.
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float* a, float* b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// One row by itself, straight from the definition: used only when a hidden
// value is not finite, where the matrix product would let it through.
template <int D>
__device__ __noinline__ void attend_row(const AttnArgs& a, int b, int hk, int head, int tok, int p) {
    const int lg = 31 - __clz(a.kv.page_size);
    const uint16_t* q = a.q + tok * a.q_tok + head * a.q_head;
    const KeyBlocks kb = key_blocks<16>(p, p, a.window, a.sinks);
    float m = kNegInf, l = 0.f;
    for (int d0 = -32; d0 < D; d0 += 32) {          // first pass: m and l; then 32 columns a pass
        float o[32];
        for (int i = 0; i < 32; ++i) o[i] = 0.f;
        for (int c = 0; c < kb.n * 16; ++c) {
            const int j = kb(c >> 4) * 16 + (c & 15);
            if (!key_visible(j, p, a.window, a.sinks)) continue;
            const int page = page_of(a.kv, b, j >> lg, a.err), slot = j & (a.kv.page_size - 1);
            const uint16_t* k = a.kv.k + page * a.kv.k_page_stride + hk * a.kv.k_head_stride + slot * a.kv.k_slot_stride;
            float s = 0.f;
            for (int d = 0; d < D; ++d) s = fmaf(bf16_bits_to_f32(q[d]), bf16_bits_to_f32(k[d]), s);
            if (d0 < 0) {
                const float mn = fmaxf(m, s);
                l = l * (mn == m ? 1.f : ex2_approx((m - mn) * a.scale)) + ex2_approx((s - mn) * a.scale);
                m = mn;
            } else {
                const uint16_t* v = a.kv.v + page * a.kv.v_page_stride + hk * a.kv.v_head_stride +
                                    slot * a.kv.v_slot_stride + d0;
                const float w = ex2_approx((s - m) * a.scale) / l;
                for (int i = 0; i < 32; ++i) o[i] = fmaf(w, bf16_bits_to_f32(v[i]), o[i]);
            }
        }
        if (d0 >= 0)
            for (int i = 0; i < 32; ++i) a.out[((size_t)tok * a.Hq + head) * D + d0 + i] = f32_to_bf16_bits(o[i]);
    }
    if (a.lse) a.lse[(size_t)tok * a.Hq + head] = l == 0.f ? kNegInf : (m * a.scale + log2f(l)) * 0.6931471805599453f;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
k_attn_prefill(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const AttnArgs a, const int tpt) {
    constexpr int NS = slots<D>(), SB = slot_bytes<D>();
    constexpr uint32_t IDESC_S = idesc_bf16_f32(kTile, kN);
    constexpr uint32_t IDESC_O = idesc_bf16_f32(kTile, D) | (1u << 16);      // B is MN major
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    uint8_t* qs = base;                                   // [2][D/64 panels][128 rows][128 B]
    uint8_t* ring = qs + 2 * kTile * D * 2;
    Ctl* ctl = reinterpret_cast<Ctl*>(ring + NS * SB);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_wait();
    pdl_launch();
    // ---- this CTA's tiles: the last tokens of every sequence first (under a
    // causal mask they see the most keys)
    const int nbh = a.kv.batch * a.kv.heads;
    const int y = blockIdx.x / nbh, bh = blockIdx.x - y * nbh;
    const int b = bh / a.kv.heads, hk = bh - b * a.kv.heads;
    const int g = a.Hq / a.kv.heads;
    int t0, t1;
    seq_rows(a.goff, b, a.T, &t0, &t1, a.err);
    const int nq = t1 - t0;
    if (nq > a.max_q) {
        if (threadIdx.x == 0) atomicCAS(a.err, 0, W4_ERR_GROUP_TOKENS);
        return;
    }
    const int pairs = (nq + 2 * tpt - 1) / (2 * tpt);
    if (y >= pairs) return;
    const int i0 = (pairs - 1 - y) * 2 * tpt;             // first token of tile A in the sequence
    const int n_tok = min(nq - i0, 2 * tpt);
    const int ntile = n_tok > tpt ? 2 : 1;
    const int len = kv_length(a.kv, b, a.max_len, a.err);
    const int p0 = len - nq + i0, p1 = p0 + n_tok - 1;    // positions of the first and last token
    const KeyBlocks kb = key_blocks<kN>(max(p0, 0), p1, a.window, a.sinks);
    // row r of tile x: token i0 + x tpt + r / g, query head hk g + r % g
    const int tile = warp >> 2;                           // of a softmax warp
    const int r = threadIdx.x & 127, rt = r / g;
    const int tok_in = tile * tpt + rt;
    const bool have = warp < 8 && rt < tpt && tok_in < n_tok;
    const int tok = t0 + i0 + tok_in, head = hk * g + (r - rt * g);
    const int p = have ? p0 + tok_in : -1;
    uint16_t* orow = a.out + ((size_t)tok * a.Hq + head) * D;
    if (kb.n == 0) {                                      // no row sees a key
        if (have) {
            for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(orow + d) = make_uint4(0, 0, 0, 0);
            if (a.lse) a.lse[(size_t)tok * a.Hq + head] = kNegInf;
        }
        return;
    }
    // block j0 is seen entirely by every row
    auto all_see = [&](int j0) {
        return j0 + kN - 1 <= p0 && (a.window == 0 || p1 - j0 < a.window || j0 + kN <= a.sinks);
    };

    if (threadIdx.x == 0) {
        mbar_init(&ctl->qfull, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
            mbar_init(&ctl->vready[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->sfull[i], 1);
            mbar_init(&ctl->pready[i], 4);
            mbar_init(&ctl->ofull[i], 1);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        ctl->bad = 0;
        fence_mbar_init();
    }
    if (warp == 9) { tmem_alloc(&ctl->tmem, 512); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    auto s_col = [&](int x) { return tmem + (uint32_t)(x * kN); };
    auto o_col = [&](int x) { return tmem + (uint32_t)(2 * kN + x * D); };
    volatile int* abort = &ctl->abort;

    // the registers of 384 threads x 168: two softmax groups of 208, one of 88
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8) {
            // -------------------------------------------------------- TMA
            const int lg = 31 - __clz(a.kv.page_size);
            const int R = min(a.kv.page_size, kN), npg = kN / R;
            if (lane == 0) {
                mbar_arrive_expect_tx(&ctl->qfull, (uint32_t)(ntile * tpt * g * D * 2));
                for (int x = 0; x < ntile; ++x)
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(qs + (x * (D / 64) + c) * kTile * 128, &tmQ, c * 64, hk * g, t0 + i0 + x * tpt,
                                    &ctl->qfull);
            }
            __syncwarp();
            uint32_t it = 0;
            bool ok = true;
            for (int c = 0; c < kb.n && ok; ++c) {
                const int j0 = kb(c) * kN;
                // lane: page pg of the block, 64-column panel pn; a page past the end is out of bounds
                const int pg = lane % npg, pn = lane / npg, jp = j0 + pg * R;
                int page = a.kv.pages;
                if (pn < D / 64 && jp < len) page = page_of(a.kv, b, jp >> lg, a.err);
                for (int kv = 0; kv < 2 && ok; ++kv, ++it) {
                    const int st = it % NS;
                    if (it >= (uint32_t)NS)
                        ok = __all_sync(0xffffffffu, mbar_wait(&ctl->empty[st], ((it / NS) & 1) ^ 1, abort, a.err));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], SB);
                    __syncwarp();
                    if (pn < D / 64)
                        tma_load_4d(ring + st * SB + pn * kN * 128 + pg * R * 128, kv ? &tmV : &tmK, pn * 64,
                                    jp & (a.kv.page_size - 1), hk, page, &ctl->full[st]);
                }
            }
            if (lane == 0) {                              // every copy lands before the CTA ends
                mbar_wait_drain(&ctl->qfull, 0, a.err);
                for (uint32_t j = it > (uint32_t)NS ? it - NS : 0; j < it; ++j)
                    mbar_wait_drain(&ctl->full[j % NS], (j / NS) & 1, a.err);
            }
        } else if (warp == 9) {
            // -------------------------------------------------------- MMA
            if (lane == 0) {
                auto mma_s = [&](int x, int st) {         // S_x = Q_x K^T
                    const uint32_t q = smem_u32(qs + x * (D / 64) * kTile * 128), k = smem_u32(ring + st * SB);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t off = (i >> 2) * kTile * 128 + (i & 3) * 32;
                        tc_mma_f16(s_col(x), smem_desc_sw128(q + off), smem_desc_sw128(k + off), IDESC_S, i > 0);
                    }
                };
                auto mma_o = [&](int x, int st, bool acc) {   // O_x += P_x V
                    const uint32_t v = smem_u32(ring + st * SB);
#pragma unroll
                    for (int i = 0; i < kN / 16; ++i)
                        tc_mma_f16_ta(o_col(x), s_col(x) + 8 * i, smem_desc_mn_sw128(v + i * 2048, kN * 128), IDESC_O,
                                      acc || i > 0);
                };
                bool ok = mbar_wait(&ctl->qfull, 0, abort, a.err) && mbar_wait(&ctl->full[0], 0, abort, a.err);
                if (ok) {
                    tc_fence_after();
                    for (int x = 0; x < ntile; ++x) { mma_s(x, 0); tc_commit(&ctl->sfull[x]); }
                    tc_commit(&ctl->empty[0]);
                }
                for (int c = 0; c < kb.n && ok; ++c) {
                    const uint32_t iv = 2 * c + 1, ik = 2 * c + 2;      // ring items of V c and K c + 1
                    const int sv = iv % NS, sk = ik % NS;
                    const bool more = c + 1 < kb.n;
                    for (int x = 0; x < ntile && ok; ++x) {
                        ok = mbar_wait(&ctl->pready[x], c & 1, abort, a.err) &&
                             (x > 0 || mbar_wait(&ctl->vready[sv], (iv / NS) & 1, abort, a.err));
                        if (!ok) break;
                        tc_fence_after();
                        mma_o(x, sv, c > 0);
                        if (x == ntile - 1) tc_commit(&ctl->empty[sv]);
                        if (!more) { tc_commit(&ctl->ofull[x]); continue; }
                        if (x == 0) {
                            ok = mbar_wait(&ctl->full[sk], (ik / NS) & 1, abort, a.err);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        mma_s(x, sk);
                        tc_commit(&ctl->sfull[x]);
                        if (x == ntile - 1) tc_commit(&ctl->empty[sk]);
                    }
                }
                // every MMA completes before the CTA ends
                tc_commit(&ctl->drain);
                mbar_wait_drain(&ctl->drain, 0, a.err);
            }
        } else {
            // -------------------------------------------------------- V release
            for (int c = 0; c < kb.n; ++c) {
                const uint32_t iv = 2 * c + 1;
                const int st = iv % NS, j0 = kb(c) * kN;
                if (!__all_sync(0xffffffffu, mbar_wait(&ctl->full[st], (iv / NS) & 1, abort, a.err))) break;
                if (!all_see(j0)) {
                    uint8_t* v = ring + st * SB;
                    bool bad = false;
                    // 16-byte pieces: panel, row, piece (the swizzle only permutes a row's pieces)
                    for (int i = (warp - 10) * 32 + lane; i < kN * D / 8; i += 64) {
                        uint4* w = reinterpret_cast<uint4*>(v) + i;
                        const int j = j0 + ((i >> 3) & (kN - 1));
                        if (j >= len) {
                            *w = make_uint4(0, 0, 0, 0);
                        } else {
                            const uint4 u = *w;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t z = (&u.x)[e];
                                bad |= (z & 0x7F80u) == 0x7F80u || (z & 0x7F800000u) == 0x7F800000u;
                            }
                        }
                    }
                    if (bad) *(volatile int*)&ctl->bad = 1;
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->vready[st]);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        if (tile < ntile) {
            const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_addr = s_col(tile) + lane_base, o_addr = o_col(tile) + lane_base;
            const float sc = a.scale;
            float m = kNegInf, l = 0.f;
            bool ok = true;
            for (int c = 0; c < kb.n; ++c) {
                ok = __all_sync(0xffffffffu, mbar_wait(&ctl->sfull[tile], c & 1, abort, a.err));
                if (!ok) break;
                tc_fence_after();
                uint32_t su[kN];
#pragma unroll
                for (int i = 0; i < kN / 32; ++i) tmem_ld_32x32b_x32(s_addr + 32 * i, su + 32 * i);
                float* s = reinterpret_cast<float*>(su);
                const int j0 = kb(c) * kN;
                if (!all_see(j0)) {
                    const int hi = p - j0, lo = a.window ? hi - a.window + 1 : -(1 << 30), sk = a.sinks - j0;
#pragma unroll
                    for (int i = 0; i < kN; ++i)
                        s[i] = i <= hi && (i >= lo || i < sk) ? s[i] : kNegInf;
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < kN; i += 4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[i + e]);
                const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                // S complete means this tile's O of the step before is complete too
                if (__any_sync(0xffffffffu, (mn - m) * sc > kLazy)) {
                    const float f = mn == m ? 1.f : ex2_approx((m - mn) * sc);
                    m = mn;
                    l *= f;
                    if (c > 0) {
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(o_addr + 16 * i, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st_x16(o_addr + 16 * i, o);
                        }
                    }
                }
                const float off = m == kNegInf ? 0.f : -m * sc;
                const uint64_t sc2 = pack2(sc, sc), off2 = pack2(off, off);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < kN / 32; ++i) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float x, z;
                        unpack2(fma2(pack2(s[32 * i + 2 * e], s[32 * i + 2 * e + 1]), sc2, off2), &x, &z);
                        x = ex2_approx(x);
                        z = ex2_approx(z);
                        sum[e & 1] = add2(sum[e & 1], pack2(x, z));
                        pk[e] = pack_bf16x2(x, z);
                    }
                    tmem_st_x16(s_addr + 16 * i, pk);
                }
                float x, z;
                unpack2(add2(sum[0], sum[1]), &x, &z);
                l += x + z;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->pready[tile]);
            }
            // -------------------------------------------------------- epilogue
            if (ok && __all_sync(0xffffffffu, mbar_wait(&ctl->ofull[tile], 0, abort, a.err))) {
                tc_fence_after();
                if (*(volatile int*)&ctl->bad) {
                    if (have && p >= 0) attend_row<D>(a, b, hk, head, tok, p);
                    else if (have) {
                        for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(orow + d) = make_uint4(0, 0, 0, 0);
                        if (a.lse) a.lse[(size_t)tok * a.Hq + head] = kNegInf;
                    }
                } else {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(o_addr + 32 * i, o);
                        if (have) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    w[z] = pack_bf16x2(__uint_as_float(o[e + 2 * z]) * inv,
                                                       __uint_as_float(o[e + 2 * z + 1]) * inv);
                                *reinterpret_cast<uint4*>(orow + 32 * i + e) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                    if (have && a.lse)
                        a.lse[(size_t)tok * a.Hq + head] = l == 0.f ? kNegInf : (m * sc + log2f(l)) * 0.6931471805599453f;
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

bool encode_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box) {
    return encode_tmap_nd(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rank, dims, strides, box,
                          CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D>
int go(const AttnArgs& a, cudaStream_t stream) {
    const int g = a.Hq / a.kv.heads, tpt = kTile / g;
    const uint32_t R = (uint32_t)std::min(a.kv.page_size, kN);
    CUtensorMap tmQ, tmK, tmV;
    const uint64_t qd[3] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.T};
    const uint64_t qst[2] = {(uint64_t)a.q_head * 2, (uint64_t)a.q_tok * 2};
    const uint32_t qb[3] = {64, (uint32_t)g, (uint32_t)tpt};
    const uint64_t kd[4] = {(uint64_t)D, (uint64_t)a.kv.page_size, (uint64_t)a.kv.heads, (uint64_t)a.kv.pages};
    const uint64_t ks[3] = {(uint64_t)a.kv.k_slot_stride * 2, (uint64_t)a.kv.k_head_stride * 2,
                            (uint64_t)a.kv.k_page_stride * 2};
    const uint64_t vs[3] = {(uint64_t)a.kv.v_slot_stride * 2, (uint64_t)a.kv.v_head_stride * 2,
                            (uint64_t)a.kv.v_page_stride * 2};
    const uint32_t kbx[4] = {64, R, 1, 1};
    if (!encode_map(&tmQ, a.q, 3, qd, qst, qb) || !encode_map(&tmK, a.kv.k, 4, kd, ks, kbx) ||
        !encode_map(&tmV, a.kv.v, 4, kd, vs, kbx))
        return W4_ERR_CUDA;
    const long long grid = ((long long)a.max_q + 2 * tpt - 1) / (2 * tpt) * a.kv.batch * a.kv.heads;
    if (grid > 0x7fffffffLL) return W4_ERR_UNSUPPORTED_SHAPE;
    constexpr size_t bytes = smem_total<D>();
    if (cudaFuncSetAttribute(k_attn_prefill<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return W4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attn_prefill<D>, tmQ, tmK, tmV, a, tpt) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

}  // namespace

size_t attn_prefill_ws_bytes(int, int, int, int, int, int, int) { return 0; }

int launch_attn_prefill(const AttnArgs& a, int, cudaStream_t stream) {
    return a.kv.head_dim == 128 ? go<128>(a, stream) : go<64>(a, stream);
}

}  // namespace w4
