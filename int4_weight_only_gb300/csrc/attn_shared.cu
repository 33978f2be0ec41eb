// attn_shared.cu - attention of one new token where groups of sequences share
// their first tokens: the keys that each sequence has of its own, and the join.
//
//   softmax over the shared and the own keys = parts (m, l, o) over any runs of
//   them, joined by  m = max m_i,  l = sum e^(m_i - m) l_i,  o = sum e^(m_i - m) o_i
//
// Three kernels: the own keys, the shared keys (attn_prefill.cu: the sequences of a group are the
// rows of tensor-core tiles, so that a key is read once for all of them) and the join.  Own keys are many short pieces (a question behind a document), where
// what counts is latency: in k_attn_decode's form, a CTA's eight warps meeting at every
// item's end, 256 sequences of 1 to 2000 own keys (125 MB, 18 us of reading) took 77 us with
// their join.  So here a warp is a worker of its own.  The list of all items' 16-key blocks
// (and kOwnUnits an item for starting and finishing one) is cut into equal consecutive
// shares, one per warp; a warp's ring of blocks runs on across the end of an item, it meets no
// barrier, and writes each part of an item as fp32 rows straight from its registers.
//
// The own keys come first.  The kernel of the shared keys needs nothing of them, so it begins
// on SMs that have finished theirs while others still work on them: the first kernel lets it
// start only once all that precedes the call is complete, and it waits for the first at its end,
// so that the join sees both.  The join then finds the shared keys' parts, which are more, in L2
// (64 sequences behind 32768 tokens 55.1 us, in the other order 56.8).
//
// The join is one to eight warps a row (sequence, head).  Parts are added in an order that
// depends on the inputs' shapes alone: the same inputs give the same bits.
//
// Measured (28 / 4 heads of 128, in a graph, own keys 1 to 2000): 256 sequences behind 32768
// shared tokens 143 us, of which the shared keys take 105 (1140 TFLOP/s: two tiles' steps of
// 1.95 us), the own keys about 28 (two thirds of the measured copy rate) and the join 10.
// 64 behind 32768 55 us, 8 behind 8192 21.5, 4 behind 1024 14 (latency of the three kernels).
#include "attn_device.cuh"
#include "w4_internal.h"

#include <algorithm>

namespace w4 {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kOwnUnits = 1;            // what starting and finishing an item costs, in blocks
constexpr int kMinShare = 2;            // blocks that are worth a part of their own

template <int D, int NT> struct Shape {
    static constexpr int warps = D == 64 && NT == 1 ? 16 : 8;
    static constexpr int threads = 32 * warps;
    static constexpr int heads = 8 * NT;                    // query heads per item
    static constexpr int stage_bytes = 16 * D * 2 * 2;      // 16 keys, K and V
    static constexpr int stages = 192 * 1024 / warps / stage_bytes;
    static constexpr size_t smem = 1024 + (size_t)warps * stages * stage_bytes;
};

// The group of a sequence, walked upwards.
struct Group {
    int i, end, len;                    // number, end of its sequences, shared keys

    __device__ __forceinline__ void read(const SharedArgs& a) {
        const long long cap = min((long long)a.kv.max_pages * a.kv.page_size, (long long)a.max_len);
        const bool in = i >= 0 && i < a.sh.groups;
        end = i >= a.sh.groups ? 0x7fffffff : __ldg(a.sh.group + i + 1);
        len = in ? (int)min(max((long long)__ldg(a.sh.shared + i), 0LL), cap) : 0;
    }
    // the last group that begins at or before sequence b: -1 before all of them, `groups` behind
    __device__ __forceinline__ void find(const SharedArgs& a, int b) {
        int lo = -1, hi = a.sh.groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.sh.group + mid) <= b) lo = mid; else hi = mid;
        }
        i = lo;
        read(a);
        if (b >= end) next(a, b);
    }
    __device__ __forceinline__ void next(const SharedArgs& a, int b) {
        while (b >= end && i < a.sh.groups) { ++i; read(a); }
    }
    __device__ __forceinline__ int at(const SharedArgs& a, int b) {
        if (b >= end) next(a, b);
        return len;
    }
};

// A worker's part of an item.
struct Part {
    int b, it, len, lo;     // sequence, item of it, keys, first own key
    int base, units;        // the sequence's first unit in the list, units of an item
    int U, end;             // the item's first unit, end of the part
    int j0, nb, issued;     // first block (absolute), blocks, those whose copies are on their way
    int page;               // page of the next one
};

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::threads, 1)
k_shared_own(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const SharedArgs a) {
    using S = Shape<D, NT>;
    constexpr int W = S::warps, NS = S::stages, HP = S::heads;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[W][NS];
    __shared__ int s_abort, s_sum[32], s_b[W], s_base[W];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* ring = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw)) + warp * NS * S::stage_bytes;
    const int Hkv = a.kv.heads, g = a.Hq / Hkv, ngrp = (g + HP - 1) / HP, items = Hkv * ngrp, B = a.kv.batch;
    if (lane == 0) {
        for (int i = 0; i < NS; ++i) mbar_init(&full[warp][i], 1);
        fence_mbar_init();
        s_b[warp] = -1;
        if (warp == 0) { s_abort = 0; tma_prefetch_desc(&tmK); tma_prefetch_desc(&tmV); }
    }
    pdl_wait();
    pdl_launch();

    // ---- the list: a thread takes a run of sequences
    auto len_of = [&](int b) { return kv_length(a.kv, b, a.max_len, a.err); };
    auto units_of = [&](int len, int lo) { return len > lo ? (len - 1) / 16 + 1 - lo / 16 + kOwnUnits : 0; };
    const int each = (B + S::threads - 1) / S::threads, b0 = min(tid * each, B), b1 = min(b0 + each, B);
    Group grp;
    int sum = 0;
    if (b0 < b1) {
        grp.find(a, b0);
        for (int b = b0; b < b1; ++b) sum += items * units_of(len_of(b), grp.at(a, b));
    }
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kAll, scan, o);
        if (lane >= o) scan += t;
    }
    if (lane == 31) s_sum[warp] = scan;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    const int first = before + scan - sum;              // of the thread's sequences
    const int share = max((total + (int)gridDim.x * W - 1) / ((int)gridDim.x * W), kMinShare);
    const int w0 = (int)blockIdx.x * W;
    const bool publish = blockIdx.x == 0;
    if (publish && tid == 0) *a.sh.own_share = share;
    if (b0 < b1 && (publish || (first < share * (w0 + W) && first + sum > share * w0))) {
        grp.find(a, b0);
        int at = first;
        for (int b = b0; b < b1; ++b) {
            const int u = units_of(len_of(b), grp.at(a, b)), n = items * u;
            if (publish) a.sh.own_info[b] = make_int2(at, u);
            // the workers whose shares begin in this sequence
            for (int w = max((at + share - 1) / share, w0); w < w0 + W && share * w < at + n; ++w) {
                s_b[w - w0] = b;
                s_base[w - w0] = at;
            }
            at += n;
        }
    }
    __syncthreads();

    const int worker = w0 + warp, u0 = share * worker, u1 = min(u0 + share, total);
    const int lg = 31 - __clz(a.kv.page_size);
    const int ki = lane & 3, kj = lane >> 2, pj = (kj >> 1) + 4 * (kj & 1);
    const float sc = a.scale;
    auto page_at = [&](const Part& s, int i) { return i < s.nb ? page_of(a.kv, s.b, ((s.j0 + i) * 16) >> lg, a.err) : 0; };
    // the part of sequence s.b's items that starts at unit u (offsets that decrease can make the list and
    // this walk differ: the item stays one of the sequence's, and blocks stay inside it)
    auto start = [&](Part& s, int u) {
        s.it = min(max(u - s.base, 0) / s.units, items - 1);
        s.U = s.base + s.it * s.units;
        s.end = min(u1, s.U + s.units);
        const int c0 = max(u - s.U - kOwnUnits, 0), c1 = max(s.end - s.U - kOwnUnits, 0);
        s.j0 = s.lo / 16 + c0;
        s.nb = max(c1 - c0, 0);
        s.issued = 0;
        s.page = page_at(s, 0);
    };
    auto sequence = [&](Part& s, int b, int base) {
        s.b = b;
        s.base = base;
        s.len = len_of(b);
        s.lo = grp.at(a, b);
        s.units = units_of(s.len, s.lo);
    };
    auto after = [&](const Part& s) {
        Part n = s;
        if (s.end == s.base + s.units * items) {
            n.units = 0;
            while (n.units == 0 && n.b + 1 < B) sequence(n, n.b + 1, s.end);
        }
        if (n.units > 0) {
            start(n, s.end);
        } else {                                        // never, unless the lengths change meanwhile
            n.nb = n.issued = 0;
            n.end = u1;
        }
        return n;
    };
    bool ok = true;
    uint32_t put = 0, got = 0;                          // blocks issued and consumed
    if (s_b[warp] >= 0) {
        Part cur, nxt;
        grp.find(a, s_b[warp]);
        sequence(cur, s_b[warp], s_base[warp]);
        start(cur, u0);
        // query pieces: head 8 x + lane / 4; those of the next part are loaded ahead where registers allow
        constexpr bool AHEAD = NT == 1;
        auto load_q = [&](const Part& s, uint4 (&q)[NT][D / 32]) {
            const int hk = s.it / ngrp, h0 = hk * g + (s.it - hk * ngrp) * HP, rows = min(HP, (hk + 1) * g - h0);
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    q[x][c] = 8 * x + kj < rows
                        ? __ldg(reinterpret_cast<const uint4*>(a.q + s.b * a.q_tok + (h0 + 8 * x + kj) * a.q_head + c * 32 + ki * 8))
                        : make_uint4(0, 0, 0, 0);
        };
        uint4 qn[AHEAD ? NT : 1][D / 32];
        if constexpr (AHEAD) load_q(cur, qn);
        auto issue = [&](Part& s) {
            if (lane == 0) {
                uint64_t* bar = &full[warp][put % NS];
                uint8_t* dst = ring + (put % NS) * S::stage_bytes;
                const int slot = ((s.j0 + s.issued) * 16) & (a.kv.page_size - 1), hk = s.it / ngrp;
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
            auto fill = [&] {                           // keep the ring full, into the next part too
                while (ok && put - got < (uint32_t)NS) {
                    if (cur.issued < cur.nb) issue(cur);
                    else if (more && nxt.issued < nxt.nb) issue(nxt);
                    else break;
                }
            };
            fill();
            if (AHEAD && cur.nb == 0 && more) {
                if constexpr (AHEAD) load_q(nxt, qn);
            }
            if (cur.nb > 0) {
                const int hk = cur.it / ngrp, h0 = hk * g + (cur.it - hk * ngrp) * HP, rows = min(HP, (hk + 1) * g - h0);
                const int p = cur.len - 1, lo = cur.lo;
                auto seen = [&](int j) { return j <= p && j >= lo; };
                uint4 qf[NT][D / 32];
                if constexpr (AHEAD) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) qf[0][c] = qn[0][c];
                    if (more) load_q(nxt, qn);
                } else {
                    load_q(cur, qf);
                }
                // o[x][mt][e]: head 8 x + 2 ki + (e & 1), column 64 (mt / 4) + 8 pj + 2 (mt % 4) + (e >> 1)
                float o[NT][D / 16][4], m[NT][2], l[NT][2], off[NT][2];
#pragma unroll
                for (int x = 0; x < NT; ++x) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) o[x][i][0] = o[x][i][1] = o[x][i][2] = o[x][i][3] = 0.f;
                    m[x][0] = m[x][1] = kNegInf;
                    l[x][0] = l[x][1] = off[x][0] = off[x][1] = 0.f;
                }
                for (int i = 0; i < cur.nb; ++i) {
                    ok = ok && __all_sync(kAll, mbar_wait(&full[warp][got % NS], (got / NS) & 1, &s_abort, a.err));
                    if (!ok) break;
                    const int j0 = (cur.j0 + i) * 16;
                    attend_block<D, NT>(ring + (got % NS) * S::stage_bytes, qf, o, m, l, off, sc, j0, j0 + 15 <= p && j0 >= lo, seen);
                    __syncwarp();                       // the stage is read: refill it
                    ++got;
                    fill();
                }
                // ---- the part's rows
                const int one = (cur.U + cur.units - 1) / share == (cur.U + kOwnUnits) / share;
                const size_t slot = 2 * worker + (cur.U + kOwnUnits < u0 ? 0 : 1);
                float* to_o = one ? a.sh.own_row_o + ((size_t)cur.b * a.Hq + h0) * D : a.sh.own_slot_o + slot * HP * D;
                float* to_ml = one ? a.sh.own_row_ml + ((size_t)cur.b * a.Hq + h0) * 2 : a.sh.own_slot_ml + slot * HP * 2;
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = l[x][e];
#pragma unroll
                        for (int z = 4; z < 32; z <<= 1) t += __shfl_xor_sync(kAll, t, z);
                        const int h = 8 * x + 2 * ki + e;
                        if (h >= rows) continue;
                        if (kj == 0) *reinterpret_cast<float2*>(to_ml + h * 2) = make_float2(m[x][e], t);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
#pragma unroll
                            for (int z = 0; z < 4; z += 2)
                                *reinterpret_cast<float4*>(to_o + h * D + c * 64 + pj * 8 + 2 * z) = make_float4(
                                    o[x][c * 4 + z][e], o[x][c * 4 + z][e + 2], o[x][c * 4 + z + 1][e], o[x][c * 4 + z + 1][e + 2]);
                    }
            }
            if (!more) break;
            cur = nxt;
        }
        // a wait ran out: the copies already issued land before the CTA ends
        if (!ok && lane == 0)
            for (; got != put; ++got) mbar_wait_drain(&full[warp][got % NS], (got / NS) & 1, a.err);
    }
}

// The parts of one row: from the kernel of the shared keys, then of the own keys.  What the lists
// say is kept inside the scratch, whatever it holds (a refused group leaves its own unwritten).
struct RowParts {
    const float *po, *pml, *oo, *oml;   // part 0 of each
    size_t pstep, ostep;                // rows from slot to slot; 0: one part, in a row of its own
    int np, no;

    __device__ __forceinline__ size_t at(size_t step, int x) const { return x == 0 ? step : 2 * x * step; }
};

template <int D>
__device__ __forceinline__ RowParts row_parts(const SharedArgs& a, int b, int h, int HP, int workers, int ctas) {
    RowParts r{};
    const int g = a.Hq / a.kv.heads, hk = h / g, hin = h - hk * g, len = kv_length(a.kv, b, a.max_len, a.err);
    const int4 s = __ldg(a.sh.info + b);
    const int2 w = __ldg(a.sh.own_info + b);
    const int share = max(__ldg(a.sh.share), 1), own = max(__ldg(a.sh.own_share), 1);
    if (len == 0) return r;
    const size_t row = (size_t)b * a.Hq + h;
    if (s.z > kSharedItemUnits) {
        const int tpt = kSharedRows / 2 / g, u = s.y + hk * s.z, first = min(max((u + kSharedItemUnits) / share, 0), ctas - 1);
        const int place = s.w & 0xFFFF, tile = place >= tpt ? 1 : 0;
        r.np = min(max((u + s.z - (s.w >> 16)) / share - first + 1, 1), ctas - first);
        const int at = min(max(tile * (kSharedRows / 2) + (place - tile * tpt) * g + hin, 0), kSharedRows - 1);
        const size_t slot = (size_t)2 * first * kSharedRows + at;
        r.pstep = r.np == 1 ? 0 : kSharedRows;
        r.po = r.np == 1 ? a.sh.row_o + row * D : a.sh.slot_o + slot * D;
        r.pml = r.np == 1 ? a.sh.row_ml + row * 2 : a.sh.slot_ml + slot * 2;
    }
    if (w.y > kOwnUnits) {
        const int grp = hin / HP, u = w.x + (hk * ((g + HP - 1) / HP) + grp) * w.y;
        const int first = min(max((u + kOwnUnits) / own, 0), workers - 1);
        r.no = min(max((u + w.y - 1) / own - first + 1, 1), workers - first);
        const size_t slot = (size_t)2 * first * HP + (hin - grp * HP);
        r.ostep = r.no == 1 ? 0 : HP;
        r.oo = r.no == 1 ? a.sh.own_row_o + row * D : a.sh.own_slot_o + slot * D;
        r.oml = r.no == 1 ? a.sh.own_row_ml + row * 2 : a.sh.own_slot_ml + slot * 2;
    }
    return r;
}

// WPR warps a row; D / 4 lanes a part.
constexpr int kJoinThreads = 256;
template <int D, int WPR>
__global__ void __launch_bounds__(kJoinThreads) k_shared_join(const SharedArgs a, int HP, int workers, int ctas) {
    constexpr int LP = D / 4, PW = 32 / LP, RPC = kJoinThreads / 32 / WPR;       // parts a warp, rows a CTA
    __shared__ float4 s_o[WPR > 1 ? RPC * WPR : 1][LP];
    __shared__ float2 s_ml[WPR > 1 ? RPC * WPR : 1];
    pdl_wait();
    pdl_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane % LP * 4;
    const long long row = (long long)blockIdx.x * RPC + warp / WPR, rows = (long long)a.kv.batch * a.Hq;
    const float sc = a.scale;
    float m = kNegInf, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows) {
        const int b = (int)(row / a.Hq);
        const RowParts r = row_parts<D>(a, b, (int)(row - (long long)b * a.Hq), HP, workers, ctas);
        const int n = r.np + r.no;
        // Parts whose loads are in flight together.  28 / 4 heads of 128, 4 and 8 of them: 224 rows (8 warps
        // a row) 21.9 and 21.0 us a call, 896 (4) 28.4 and 27.7, but 1024 rows of 64 23.9 and 25.5,
        // 1792 (2) 55.6 and 54.5, 7168 (1) 145.8 and 147.0; 2 of them up to 2.9 us slower.
        constexpr int U = WPR == 8 || WPR == 2 ? 8 : 4;
        for (int x0 = (warp % WPR) * PW + lane / LP; x0 < n; x0 += WPR * PW * U) {
            float2 ml[U];
            float4 t[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int x = x0 + i * WPR * PW;
                const bool pre = x < r.np;
                const size_t p = pre ? r.at(r.pstep, x) : r.at(r.ostep, x - r.np);
                ml[i] = x < n ? __ldcg(reinterpret_cast<const float2*>((pre ? r.pml : r.oml) + p * 2)) : make_float2(kNegInf, 0.f);
                t[i] = x < n ? __ldcg(reinterpret_cast<const float4*>((pre ? r.po : r.oo) + p * D + col))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mx = m;
#pragma unroll
            for (int i = 0; i < U; ++i) mx = fmaxf(mx, ml[i].x);
            const float f0 = m == mx ? 1.f : ex2_approx((m - mx) * sc);
            o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
            l *= f0;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float f = ml[i].x == mx ? 1.f : ex2_approx((ml[i].x - mx) * sc);
                l += f * ml[i].y;
                o.x += f * t[i].x; o.y += f * t[i].y; o.z += f * t[i].z; o.w += f * t[i].w;
            }
            m = mx;
        }
    }
    auto add = [&](float m2, float l2, float4 o2) {
        const float mx = fmaxf(m, m2), f = m == mx ? 1.f : ex2_approx((m - mx) * sc), f2 = m2 == mx ? 1.f : ex2_approx((m2 - mx) * sc);
        l = l * f + l2 * f2;
        o.x = o.x * f + o2.x * f2; o.y = o.y * f + o2.y * f2; o.z = o.z * f + o2.z * f2; o.w = o.w * f + o2.w * f2;
        m = mx;
    };
    if constexpr (PW == 2) {
        __syncwarp();
        const float m2 = __shfl_down_sync(kAll, m, 16), l2 = __shfl_down_sync(kAll, l, 16);
        const float4 o2 = make_float4(__shfl_down_sync(kAll, o.x, 16), __shfl_down_sync(kAll, o.y, 16),
                                      __shfl_down_sync(kAll, o.z, 16), __shfl_down_sync(kAll, o.w, 16));
        add(m2, l2, o2);
    }
    if constexpr (WPR > 1) {
        if (lane < LP) s_o[warp][lane] = o;
        if (lane == 0) s_ml[warp] = make_float2(m, l);
        __syncthreads();
        if (warp % WPR || lane >= LP) return;
#pragma unroll
        for (int i = 1; i < WPR; ++i) add(s_ml[warp + i].x, s_ml[warp + i].y, s_o[warp + i][lane]);
    }
    if (row >= rows || lane >= LP) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(a.out + row * D + col) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? kNegInf : (m * sc + log2f(l)) * 0.6931471805599453f;
}

bool launch(const void* kern, long long grid, int threads, size_t smem, void** args, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, args) == cudaSuccess;
}

template <int D, int NT>
int own(SharedArgs a, int sm_count, cudaStream_t stream) {
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
    static SmemLimit limit;
    if (!limit.raise(k_shared_own<D, NT>, (int)S::smem)) return W4_ERR_CUDA;
    void* args[] = {&tmK, &tmV, &a};
    return launch((const void*)k_shared_own<D, NT>, sm_count, S::threads, S::smem, args, stream) ? W4_OK : W4_ERR_CUDA;
}

template <int D, int NT>
int join(SharedArgs a, int sm_count, cudaStream_t stream) {
    using S = Shape<D, NT>;
    int HP = S::heads, workers = sm_count * S::warps, ctas = sm_count;
    void* args[] = {&a, &HP, &workers, &ctas};
    const long long rows = (long long)a.kv.batch * a.Hq;
    // Warps a row: rows are few where their parts are many.  28 / 4 heads of 128, 1, 2, 4, 8
    // warps: 8 sequences behind 8192 tokens (224 rows) -, 23.8, 22.1, 21.1 us; 32 (896) -, 31.7,
    // 30.3, 31.5; 64 behind 32768 (1792) -, 56.8, 58.7, 61; 256 (7168) 143.7, 148.7, 152.8, 170.
    auto with = [&](const void* kern, int warps) {
        const int per = kJoinThreads / 32 / warps;
        return launch(kern, (rows + per - 1) / per, kJoinThreads, 0, args, stream) ? W4_OK : W4_ERR_CUDA;
    };
    if (rows <= 2LL * sm_count) return with((const void*)k_shared_join<D, 8>, 8);
    if (rows <= 8LL * sm_count) return with((const void*)k_shared_join<D, 4>, 4);
    if (rows <= 16LL * sm_count) return with((const void*)k_shared_join<D, 2>, 2);
    return with((const void*)k_shared_join<D, 1>, 1);
}

int head_tiles(int Hq, int Hkv) { return Hq / Hkv <= 8 ? 1 : 2; }

}  // namespace

int shared_own_slots(int Hq, int Hkv, int D, int sm_count) {
    const int nt = head_tiles(Hq, Hkv);
    return 2 * sm_count * (D == 64 && nt == 1 ? 16 : 8) * 8 * nt;
}

int launch_attn_shared_own(const SharedArgs& a, int sm_count, cudaStream_t stream) {
    const int nt = head_tiles(a.Hq, a.kv.heads);
    if (a.kv.head_dim == 128) return nt == 1 ? own<128, 1>(a, sm_count, stream) : own<128, 2>(a, sm_count, stream);
    return nt == 1 ? own<64, 1>(a, sm_count, stream) : own<64, 2>(a, sm_count, stream);
}

int launch_attn_shared_join(const SharedArgs& a, int sm_count, cudaStream_t stream) {
    const int nt = head_tiles(a.Hq, a.kv.heads);
    if (a.kv.head_dim == 128) return nt == 1 ? join<128, 1>(a, sm_count, stream) : join<128, 2>(a, sm_count, stream);
    return nt == 1 ? join<64, 1>(a, sm_count, stream) : join<64, 2>(a, sm_count, stream);
}

}  // namespace w4
