// attn_decode.cu - attention of one new token over the paged cache.
//
//   o = sum_j w_j v_j,  w = softmax over the visible j of scale (q . k_j)
//
// The call is bound by reading the visible keys and values once (4 D bytes a
// key and key-value head); the query heads of a group share that read as the
// columns of one matrix operand.
//
// Work: an item is (sequence, key-value head, group of up to 8 NT query heads),
// a unit of it 16 keys for each warp of a CTA.  Lengths are known on the device
// only.  A few items are cut into equal parts, one per CTA.  Otherwise the units
// of all items form one list, cut into equal consecutive shares, one per CTA; an
// item counts kItemUnits units more than it has keys for, which is about what
// starting and joining one costs.  An item that several CTAs work on is joined
// from fp32 partial sums by the last of them to arrive, in the order of the
// keys: the same inputs give the same bits.
//
// Both products run transposed, so that keys fill the 16-row side of
// mma.sync m16n8k16 and the few query heads its 8 columns:
//   S^T [16 keys x 8 heads] = K Q^T,   O^T [D x 8 heads] += V^T P^T
// A block is 16 keys.  Each warp has its own blocks and its own ring of
// kStages of them in shared memory, filled by one TMA each for K and V (a
// page's 16 rows, 64-column panels, 128-byte swizzle) that its first lane
// issues, also across the end of an item into the next one; no barrier is
// shared inside the loop.  Both products sum over an index whose order is free
// (the head dimension, the keys), so a lane's operand words are whole 16-byte
// pieces, read without bank conflicts (pi(x) = x / 2 + 4 (x % 2)):
//   K piece (c, h): key pi(lane / 4) + 8 h, values 32 c + 8 (lane % 4) .. + 7
//   V piece (c, n): key lane % 4 + 4 n, values 64 c + 8 pi(lane / 4) .. + 7
// Values of two keys are interleaved in registers (one byte permute a word)
// and P is transposed with movmatrix.
//
// A block is read only if the token sees some of its keys; pieces of the
// others (which may hold anything) are zeroed in registers and their scores
// masked.
//
// The running maximum is lazy: a warp keeps the maximum it scaled by until a
// score exceeds it by 2^8, so the common step has no shuffles and no rescaling.
// l sums the fp32 weights.  As matrix operands they are two bf16 values, the
// weight's upper half and what that leaves, so the values' products see 15
// bits of them: the second product costs nothing under the loads (8 sequences
// of 128k keys: 331 us with it, 330 without) and brings the output's error
// from 1.4 times that of one rounding down to it.  Both parts of a weight are
// positive, so an infinite value that the token sees gives the infinity.
//
// Measured (28 / 4 heads of 128): 8 sequences of 128k keys 331-338 us, 0.91-0.93
// of the measured copy rate; 64 ragged ones (1 to 8192 keys) 41 us, 0.68 (CTAs
// finish 33 us after the start on average); one of 517 keys 7.1 us of latency
// (lookup, first keys, join).  More than 16 heads to one key-value head are items of
// their own that read the keys again: 8 sequences of 32768 keys take 32 us for 16
// heads, 84 for 64 and 157 for 128.
#include "attn_device.cuh"
#include "w4_internal.h"

#include <algorithm>

namespace w4 {
namespace {

// What starting and joining an item costs, in units: 64 ragged sequences take 55 us
// with 0, 42 with 1, 41 with 2 and 3; uniform long ones do not depend on it.
constexpr int kItemUnits = 2;

// One CTA per SM; warps and ring depth fill its registers and shared memory.
template <int D, int NT> struct Shape {
    static constexpr int warps = D == 64 && NT == 1 ? 16 : 8;
    static constexpr int threads = 32 * warps;
    static constexpr int stages = D == 128 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 3 : 5);
    static constexpr int heads = 8 * NT;                    // query heads per item
    static constexpr int stage_bytes = 16 * D * 2 * 2;      // 16 keys, K and V
    static constexpr int ring_bytes = warps * stages * stage_bytes;
    static constexpr int orow = D + 4;                      // padded row of the warps' outputs
    // join: threads of a part: D / 4 columns x `split` shares of the heads; parts summed at a time
    static constexpr int split = warps == 16 || NT == 2 ? 4 : 2;
    static constexpr int groups = threads / (D / 4) / split;
    // the outputs of half the warps, or the sums of the join's groups
    static constexpr int join_floats =
        warps / 2 * heads * orow > groups * heads * D ? warps / 2 * heads * orow : groups * heads * D;
    // a partial result: o [heads][D], then m [heads], l [heads]
    static constexpr int slot_floats = heads * (D + 2);
    static constexpr size_t smem = 1024 + ring_bytes + (size_t)join_floats * 4;
    static_assert(smem + 2048 <= 227 * 1024, "a CTA fits the SM's shared memory");
};

// The part of an item that a CTA works on, as one of its warps sees it.
struct Part {
    KeyBlocks kb;           // the sequence's visible 16-key blocks
    int b, it, len;         // sequence, item of it, clamped length
    int units;              // of each of its items: kItemUnits without keys, then a block per warp each
    int base;               // first unit of the sequence in the list
    int first_unit, end;    // of the item; end of the part (in the list)
    int len_after;          // length of the sequence after b (loaded ahead)
    int first, n;           // the CTAs that hold parts of the item: the first, how many
    int c0, nb;             // this warp's first block, number of blocks
    int issued;             // blocks whose copies are on their way
    int page;               // page of the next one
};

// A finished head's output row (four columns) and log-sum-exp.
template <int D>
__device__ __forceinline__ void put_out(const AttnArgs& a, size_t row, int d, float4 o, float m, float l) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(a.out + row * D + d) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && d == 0) a.lse[row] = l == 0.f ? kNegInf : (m * a.scale + log2f(l)) * 0.6931471805599453f;
}

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::threads, 1)
k_attn_decode(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnArgs a) {
    using S = Shape<D, NT>;
    constexpr int W = S::warps, NS = S::stages, HP = S::heads, SF = S::slot_floats, OS = S::orow;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[W][NS];
    __shared__ int s_last, s_abort;
    __shared__ float s_m[W / 2][HP], s_l[W / 2][HP];
    uint8_t* ring0 = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    float* so = reinterpret_cast<float*>(ring0 + S::ring_bytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* ring = ring0 + warp * NS * S::stage_bytes;
    const int Hkv = a.kv.heads, g = a.Hq / Hkv, ngrp = (g + HP - 1) / HP;
    const int items = Hkv * ngrp;           // per sequence
    const int B = a.kv.batch;
    if (lane == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(&full[warp][i], 1);
        fence_mbar_init();
        if (warp == 0) { s_abort = 0; tma_prefetch_desc(&tmK); tma_prefetch_desc(&tmV); }
    }
    __syncwarp();
    pdl_wait();
    pdl_launch();

    // ---- this CTA's work (every warp finds it by itself)
    const int G = (int)gridDim.x;
    auto blocks_of = [&](int len) { return key_blocks<16>(len - 1, len - 1, a.window, a.sinks); };
    auto len_of = [&](int b) { return b < B ? kv_length(a.kv, b, a.max_len, a.err) : 0; };
    // 0 keys: a unit that writes o = 0
    auto units_of = [&](int len) { return max(1, (blocks_of(len).n + W - 1) / W); };
    auto warp_scan = [&](int v) {           // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        return v;
    };
    const int len0 = len_of(lane), real0 = lane < B ? units_of(len0) : 0;
    int total = lane < B ? items * (real0 + kItemUnits) : 0;
    for (int b = lane + 32; b < B; b += 32) total += items * (units_of(len_of(b)) + kItemUnits);
    total = __reduce_add_sync(0xffffffffu, total);
    // consecutive shares of the list
    const int share = (total + G - 1) / G;
    int u0 = share * (int)blockIdx.x, u1 = min(u0 + share, total);
    Part cur, nxt;
    cur.b = cur.base = 0;
    int part = 0;                           // > 0: units of a part, items cut one by one
    // Equal parts win for equal lengths (28 / 4 heads, 4 sequences of 1000 keys: 8.0 us
    // against 8.8 by the list, 12 of 8000 37.8 against 39.0) and cost up to 0.3 us for
    // ragged ones.  Of 17 to 32 sequences the limit leaves equal ones to the list (24 of
    // 1000: 16.9 us, cut 14.6), since ragged ones lose there (20 up to 8000: 21.4, cut 22.9).
    if (B <= 16 && B * items <= G) {
        // each lane tries a size of part, from an equal share up; the smallest whose
        // parts are no more than the CTAs wins
        const int p = max(share - kItemUnits, 1) + lane * (1 + share / 64);
        int parts = 0;
        for (int i = 0; i < B; ++i) parts += (__shfl_sync(0xffffffffu, real0, i) + p - 1) / p;
        const uint32_t fits = __ballot_sync(0xffffffffu, parts * items <= G);
        const int best = __shfl_sync(0xffffffffu, p, __ffs(fits) - 1);
        if (fits && best <= share + kItemUnits + share / 4) part = best;
    }
    if (part) {
        const int mine = (real0 + part - 1) / part * items, v = warp_scan(mine);
        const uint32_t past = __ballot_sync(0xffffffffu, v > (int)blockIdx.x);
        if (!past) return;                  // more CTAs than parts
        cur.b = __ffs(past) - 1;
        u0 = (int)blockIdx.x - __shfl_sync(0xffffffffu, v - mine, cur.b);      // part of the sequence
        cur.len = __shfl_sync(0xffffffffu, len0, cur.b);
    } else {
        if (u0 >= total) return;
        for (int b0 = 0;; b0 += 32) {
            const int len = b0 ? len_of(b0 + lane) : len0;
            const int n = b0 + lane < B ? items * (units_of(len) + kItemUnits) : 0, v = warp_scan(n);
            const uint32_t past = __ballot_sync(0xffffffffu, cur.base + v > u0);
            if (past) {
                const int f = __ffs(past) - 1;
                cur.b = b0 + f;
                cur.base += __shfl_sync(0xffffffffu, v - n, f);
                cur.len = __shfl_sync(0xffffffffu, len, f);
                break;
            }
            cur.base += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();                        // s_abort is set

    const int lg = 31 - __clz(a.kv.page_size);
    const int ki = lane & 3, kj = lane >> 2, pj = (kj >> 1) + 4 * (kj & 1);
    const float sc = a.scale;

    auto page_at = [&](const Part& s, int i) {
        return i < s.nb ? page_of(a.kv, s.b, (s.kb(s.c0 + i * W) * 16) >> lg, a.err) : 0;
    };
    // This warp's blocks of units s0 .. s1 - 1 (counted without the first kItemUnits).
    auto take = [&](Part& s, int s0, int s1) {
        s.c0 = s0 * W + warp;
        const int c1 = min(s1 * W, s.kb.n);
        s.nb = s.c0 < c1 ? (c1 - s.c0 + W - 1) / W : 0;
        s.issued = 0;
        s.page = page_at(s, 0);
    };
    // The part of sequence s.b's items that starts at unit u of the list.
    auto start = [&](Part& s, int u) {
        s.it = (u - s.base) / s.units;
        s.first_unit = s.base + s.it * s.units;
        s.end = min(u1, s.first_unit + s.units);
        s.first = (s.first_unit + kItemUnits) / share;
        s.n = (s.first_unit + s.units - 1) / share - s.first + 1;
        take(s, max(u - s.first_unit - kItemUnits, 0), max(s.end - s.first_unit - kItemUnits, 0));
    };
    auto after = [&](const Part& s) {
        Part n = s;
        if (s.end == s.base + s.units * items) {
            n.b = s.b + 1;
            n.base = s.end;
            n.len = s.len_after;
            n.kb = blocks_of(n.len);
            n.units = units_of(n.len) + kItemUnits;
            n.len_after = len_of(n.b + 1);
        }
        start(n, s.end);
        return n;
    };
    cur.kb = blocks_of(cur.len);
    cur.units = units_of(cur.len) + kItemUnits;
    if (part) {
        // the item's units in n runs equal to one, on CTAs first .. first + n - 1
        const int real = cur.units - kItemUnits;
        cur.n = (real + part - 1) / part;
        cur.it = u0 / cur.n;
        const int x = u0 - cur.it * cur.n, each = real / cur.n, rest = real - each * cur.n;
        const int s0 = x * each + min(x, rest);
        cur.first = (int)blockIdx.x - x;
        cur.first_unit = 0;
        cur.end = u1 = kItemUnits + 1;        // no list: this part and no other
        take(cur, s0, s0 + each + (x < rest ? 1 : 0));
    } else {
        cur.len_after = len_of(cur.b + 1);
        start(cur, u0);
    }
    uint32_t put = 0, got = 0;              // blocks issued and consumed by this warp
    bool ok = true;
    auto issue = [&](Part& s) {
        const int j0 = s.kb(s.c0 + s.issued * W) * 16;
        if (lane == 0) {
            uint64_t* bar = &full[warp][put % NS];
            uint8_t* dst = ring + (put % NS) * S::stage_bytes;
            const int slot = j0 & (a.kv.page_size - 1), hk = s.it / ngrp;
            mbar_arrive_expect_tx(bar, S::stage_bytes);
            tma_load_5d(dst, &tmK, 0, slot, 0, hk, s.page, bar);
            tma_load_5d(dst + 16 * D * 2, &tmV, 0, slot, 0, hk, s.page, bar);
        }
        ++put;
        ++s.issued;
        s.page = page_at(s, s.issued);
    };

    while (true) {
        const bool more = cur.end < u1;
        if (more) nxt = after(cur);
        if (cur.end - cur.first_unit <= kItemUnits) {      // no blocks, nothing to join
            if (!more) break;
            cur = nxt;
            continue;
        }
        auto fill = [&] {                   // keep the ring full, into the next segment too
            while (ok && put - got < (uint32_t)NS) {
                if (cur.issued < cur.nb) issue(cur);
                else if (more && nxt.issued < nxt.nb) issue(nxt);
                else break;
            }
        };
        fill();
        const int hk = cur.it / ngrp, h0 = hk * g + (cur.it - hk * ngrp) * HP;
        const int rows = min(HP, (hk + 1) * g - h0);
        const int p = cur.len - 1;
        auto seen = [&](int j) { return key_visible(j, p, a.window, a.sinks); };

        // ---- query pieces: head 8 x + lane / 4
        uint4 qf[NT][D / 32];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                qf[x][c] = 8 * x + kj < rows
                    ? __ldg(reinterpret_cast<const uint4*>(a.q + cur.b * a.q_tok + (h0 + 8 * x + kj) * a.q_head + c * 32 + ki * 8))
                    : make_uint4(0, 0, 0, 0);
        // accumulators: o[x][mt][e]: head 8 x + 2 ki + (e & 1), column
        // 64 (mt / 4) + 8 pj + 2 (mt % 4) + (e >> 1)
        float o[NT][D / 16][4];
        float m[NT][2], l[NT][2], off[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[x][i][0] = o[x][i][1] = o[x][i][2] = o[x][i][3] = 0.f;
            m[x][0] = m[x][1] = kNegInf;
            l[x][0] = l[x][1] = off[x][0] = off[x][1] = 0.f;
        }
        for (int i = 0; i < cur.nb; ++i) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&full[warp][got % NS], (got / NS) & 1, &s_abort, a.err));
            if (!ok) break;
            const uint8_t* st = ring + (got % NS) * S::stage_bytes;
            const int j0 = cur.kb(cur.c0 + i * W) * 16;
            const bool all = j0 + 15 <= p && (a.window == 0 || p - j0 < a.window || j0 + 16 <= a.sinks);
            attend_block<D, NT>(st, qf, o, m, l, off, sc, j0, all, seen);
            __syncwarp();                   // the stage is read: refill it
            ++got;
            fill();
        }

        // ---- join the warps: the upper half's results go through shared memory
        // into the lower half's, then the lower half's are added in warp order
        float lw[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = l[x][e];
#pragma unroll
                for (int z = 4; z < 32; z <<= 1) t += __shfl_xor_sync(0xffffffffu, t, z);
                lw[x][e] = t;
            }
        auto out_row = [&](int x, int e) { return so + ((warp % (W / 2)) * HP + 8 * x + 2 * ki + e) * OS + pj * 8; };
        auto store_o = [&] {
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (kj == 0) {
                        s_m[warp % (W / 2)][8 * x + 2 * ki + e] = m[x][e];
                        s_l[warp % (W / 2)][8 * x + 2 * ki + e] = lw[x][e];
                    }
                    float* row = out_row(x, e);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
#pragma unroll
                        for (int t = 0; t < 4; t += 2)
                            *reinterpret_cast<float4*>(row + c * 64 + 2 * t) = make_float4(
                                o[x][c * 4 + t][e], o[x][c * 4 + t][e + 2], o[x][c * 4 + t + 1][e], o[x][c * 4 + t + 1][e + 2]);
                }
        };
        if (warp >= W / 2) store_o();
        __syncthreads();
        if (warp < W / 2) {
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float m2 = s_m[warp][8 * x + 2 * ki + e], mr = fmaxf(m[x][e], m2);
                    const float f = m[x][e] == mr ? 1.f : ex2_approx((m[x][e] - mr) * sc);
                    const float f2 = m2 == mr ? 1.f : ex2_approx((m2 - mr) * sc);
                    lw[x][e] = lw[x][e] * f + s_l[warp][8 * x + 2 * ki + e] * f2;
                    m[x][e] = mr;
                    const float* row = out_row(x, e);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const float2 z = *reinterpret_cast<const float2*>(row + c * 64 + 2 * t);
                            o[x][c * 4 + t][e] = o[x][c * 4 + t][e] * f + z.x * f2;
                            o[x][c * 4 + t][e + 2] = o[x][c * 4 + t][e + 2] * f + z.y * f2;
                        }
                }
            __syncwarp();                   // s_m and s_l of this warp are read
            store_o();
        }
        __syncthreads();

        const int n = cur.n;
        // a CTA has at most two parts of items that others work on too: one that began
        // before it, one that goes on after it
        auto slot_of = [&](int x) { return a.partial + (size_t)(2 * (cur.first + x) + (x ? 0 : 1)) * SF; };
        float* mine = slot_of((int)blockIdx.x - cur.first);
        const size_t row0 = (size_t)cur.b * a.Hq + h0;
        for (int i = tid; i < rows * (D / 4); i += S::threads) {
            const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
            float mr = kNegInf, lr = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < W / 2; ++x) mr = fmaxf(mr, s_m[x][r]);
#pragma unroll
            for (int x = 0; x < W / 2; ++x) {
                const float mw = s_m[x][r], f = mw == mr ? 1.f : ex2_approx((mw - mr) * sc);
                const float4 t = *reinterpret_cast<const float4*>(so + (x * HP + r) * OS + d);
                lr += f * s_l[x][r];
                v.x += f * t.x; v.y += f * t.y; v.z += f * t.z; v.w += f * t.w;
            }
            if (n == 1) {
                put_out<D>(a, row0 + r, d, v, mr, lr);
            } else {
                *reinterpret_cast<float4*>(mine + r * D + d) = v;
                if (d == 0) { mine[HP * D + r] = mr; mine[HP * D + HP + r] = lr; }
            }
        }
        if (n > 1) {
            __syncthreads();
            if (tid == 0) {
                const bool is_last = atom_add_acq_rel_gpu(a.tickets + cur.first, 1) == n - 1;
                if (is_last) a.tickets[cur.first] = 0;
                s_last = is_last;
            }
            __syncthreads();
            if (s_last) {
                // the heads' maxima and sums, then the weighted sums of the parts, the
                // thread groups taking parts in turn, their sums added in group order
                for (int r = warp; r < rows; r += W) {
                    float mr = kNegInf, lr = 0.f;
                    for (int i = lane; i < n; i += 32) {
                        const float* s = slot_of(i) + HP * D + r;
                        const float mi = __ldcg(s), li = __ldcg(s + HP), mx = fmaxf(mr, mi);
                        lr = lr * (mr == mx ? 1.f : ex2_approx((mr - mx) * sc)) +
                             li * (mi == mx ? 1.f : ex2_approx((mi - mx) * sc));
                        mr = mx;
                    }
                    float mx = mr;
#pragma unroll
                    for (int z = 16; z; z >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, z));
                    lr = warp_sum(lr * (mr == mx ? 1.f : ex2_approx((mr - mx) * sc)));
                    if (lane == 0) { s_m[0][r] = mx; s_l[0][r] = lr; }
                }
                __syncthreads();
                constexpr int HH = HP / S::split;
                const int col = (tid % (D / 4)) * 4, h1 = tid / (D / 4) % S::split * HH, grp = tid / (D / 4) / S::split;
                float4 acc[HH];
                float mh[HH];
#pragma unroll
                for (int r = 0; r < HH; ++r) {
                    acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                    mh[r] = h1 + r < rows ? s_m[0][h1 + r] : 0.f;
                }
                constexpr int U = 24 / HH;          // parts whose loads are in flight together
                for (int i0 = grp; i0 < n; i0 += U * S::groups) {
                    float4 t[U][HH];
                    float mi[U][HH];
#pragma unroll
                    for (int x = 0; x < U; ++x) {
                        const int i = i0 + x * S::groups;
                        const float* s = slot_of(min(i, n - 1));
#pragma unroll
                        for (int r = 0; r < HH; ++r) {
                            const bool in = h1 + r < rows && i < n;
                            mi[x][r] = in ? __ldcg(s + HP * D + h1 + r) : kNegInf;
                            t[x][r] = in ? __ldcg(reinterpret_cast<const float4*>(s + (h1 + r) * D + col))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    }
#pragma unroll
                    for (int x = 0; x < U; ++x)
#pragma unroll
                        for (int r = 0; r < HH; ++r) {
                            const float f = mi[x][r] == mh[r] ? 1.f : ex2_approx((mi[x][r] - mh[r]) * sc);
                            acc[r].x += f * t[x][r].x; acc[r].y += f * t[x][r].y;
                            acc[r].z += f * t[x][r].z; acc[r].w += f * t[x][r].w;
                        }
                }
#pragma unroll
                for (int r = 0; r < HH; ++r)
                    *reinterpret_cast<float4*>(so + (grp * HP + h1 + r) * D + col) = acc[r];
                __syncthreads();
                for (int i = tid; i < rows * (D / 4); i += S::threads) {
                    const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < S::groups; ++x) {
                        const float4 t = *reinterpret_cast<const float4*>(so + (x * HP + r) * D + d);
                        v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
                    }
                    put_out<D>(a, row0 + r, d, v, s_m[0][r], s_l[0][r]);
                }
            }
        }
        if (!more) break;
        __syncthreads();
        cur = nxt;
    }
    // a wait ran out: the copies already issued land before the CTA ends
    if (!ok && lane == 0)
        for (; got != put; ++got) mbar_wait_drain(&full[warp][got % NS], (got / NS) & 1, a.err);
}

template <int D, int NT>
int go(const AttnArgs& a, int sm_count, cudaStream_t stream) {
    using S = Shape<D, NT>;
    CUtensorMap tmK, tmV;
    const uint64_t dims[5] = {64, (uint64_t)a.kv.page_size, D / 64, (uint64_t)a.kv.heads, (uint64_t)a.kv.pages};
    const uint64_t ks[4] = {(uint64_t)a.kv.k_slot_stride * 2, 128, (uint64_t)a.kv.k_head_stride * 2,
                            (uint64_t)a.kv.k_page_stride * 2};
    const uint64_t vs[4] = {(uint64_t)a.kv.v_slot_stride * 2, 128, (uint64_t)a.kv.v_head_stride * 2,
                            (uint64_t)a.kv.v_page_stride * 2};
    const uint32_t box[5] = {64, 16, D / 64, 1, 1};
    if (!encode_tmap_nd(&tmK, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv.k, 5, dims, ks, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_nd(&tmV, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv.v, 5, dims, vs, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return W4_ERR_CUDA;
    const int grid = sm_count, bytes = (int)S::smem;
    static SmemLimit limit;
    if (!limit.raise(k_attn_decode<D, NT>, bytes)) return W4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(S::threads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_attn_decode<D, NT>, tmK, tmV, a) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

// Two tiles of 8 heads share the keys and values that one would read twice.
int head_tiles(int Hq, int Hkv) { return Hq / Hkv <= 8 ? 1 : 2; }

}  // namespace

size_t attn_decode_ws_bytes(int Hq, int Hkv, int D, int sm_count) {
    return (size_t)sm_count * 2 * 8 * head_tiles(Hq, Hkv) * (D + 2) * sizeof(float);
}

int launch_attn_decode(const AttnArgs& a, int sm_count, cudaStream_t stream) {
    const int nt = head_tiles(a.Hq, a.kv.heads);
    if (a.kv.head_dim == 128) return nt == 1 ? go<128, 1>(a, sm_count, stream) : go<128, 2>(a, sm_count, stream);
    return nt == 1 ? go<64, 1>(a, sm_count, stream) : go<64, 2>(a, sm_count, stream);
}

}  // namespace w4
