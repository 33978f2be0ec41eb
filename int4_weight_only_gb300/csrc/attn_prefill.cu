// attn_prefill.cu - attention of a prompt, or of a chunk behind a cached
// prefix, over the paged cache (the rule of attn_decode.cu for every token),
// on the 5th-generation tensor cores.
//
//   S = Q K^T,  P = exp2(c S - c m),  O = P V / sum(P)
//
// A query tile is 128 rows (tokens x query heads of one key-value head, so the
// heads of a group share the keys and values), a step 128 keys.  An item is two
// neighbouring tiles A and B over the same keys: while the tensor cores compute
// one tile's S and O, the other tile's warps take its exponentials.
//
// Work: one CTA per SM.  Many items: each CTA takes whole items, those with the
// most steps first (under a causal mask a sequence's last tokens), in turns that
// alternate direction, so that the sums balance.  Few items, or a few more than
// one turn: the CTAs of a thread-block cluster share an item's steps; at its end
// each writes its partial O, m and l by rows into the shared memory of the
// others, and each joins its own share of the rows, in the order of the keys.
// Either way the same inputs give the same bits.
//
// TMEM (512 columns): S_A, S_B (128 each), O_A, O_B (D each).  P is written as
// bf16 over the S it came from and is the next product's A operand, straight
// from TMEM; O is accumulated in TMEM over all steps.
//
// The running maximum m is lazy: a row keeps the maximum it scaled by until a
// step exceeds it by more than 2^8, so O is rescaled in the first steps and
// then hardly ever; P stays below 2^8, which costs bf16 nothing.  The sums use
// the fp32 weights, before they are rounded to bf16 as matrix operands: one word,
// because a second one for the rounding's rest, as in attn_decode.cu, is another
// value product where the tensor cores are the scarce part (the output is 0.0022
// from 64 bits, against 0.0016 of one rounding of the result).
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax of tile A, B (one row per thread), O to memory
//   warp 8          TMA: Q of an item, then K and V blocks into a ring of slots
//                   (K in even, V in odd slots), one box per page and 64
//                   columns; pages that hold no key a row sees are read out
//                   of bounds of the tensor map, which fills them with zeros.
//                   It runs ahead into the next item
//   warp 9          TMEM allocation; issues the MMAs, for each step
//                   O_A += P_A V, S_A = Q_A K', O_B += P_B V, S_B = Q_B K'
//   warps 10, 11    release V blocks to the MMAs.  In a block that not every
//                   row sees entirely, a weight of zero does not make a NaN
//                   harmless: slots past the end are zeroed, and a NaN or
//                   infinity in a slot that some row does not see is taken out
//                   and added at the part's end to the rows that see it
//                   (add_non_finite)
// Every wait is bounded (mbar_wait); copies and MMAs in flight are drained
// before the CTA ends.
//
// Measured (28 / 4 heads of 128, in a graph): 8192 tokens 352-358 us, 1345-1368
// TFLOP/s (347 with its exponentials left out); 2048 behind 14336 345 us; 2048
// tokens 38.2-38.6 us.  A step of two tiles takes 3330 cycles.  Its MMAs need 2048,
// and shared memory as many (128 KB for the score products' operands, 64 KB for the
// value products', 64 KB of copies, at 128 bytes a cycle): by the counters both
// are busy for 61 % of the time, and neither is the limit.  The other 1300 cycles
// are waits between a tile's score product, its softmax and its value product that
// the other tile's work does not fill.  Heads of 64 are bound by that chain alone: a
// step takes 1.46 us with two tiles, 1.20 with one.  P in TMEM columns of its
// own, which they have room for, so that the next score product starts as soon
// as S is read, took 1.63: the two tiles then run their softmax at one time.
// Uneven batches are far slower than their work: items are dealt out by position, as if
// every sequence were as long as the longest (28 / 4 heads: one prompt of 8192 tokens
// with 37 of 16 takes 6.2 ms, with 255 single tokens 1.5 ms, alone 0.35).
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
    uint64_t qfull, qempty;
    uint64_t full[8], empty[8], vready[8];
    uint64_t sfull[2], pready[2][2], ofull[2], oempty[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    // by V-releasing warp: the last part (counted from 1) with a slot that some row does not
    // see and that held a non-finite value.  Written before the V block is released, so a
    // tile that has its O finds its part's number here, or a later part's (a tile may
    // be any number of parts behind: those of one tile do not wait for the other):
    // looking through its slots then adds nothing
    int bad[2];
};

// The join of an item's parts, over the space of Q and the ring: rows of o by
// tile, part and row of this CTA's share, padded so that a warp's rows fall into
// different banks; then m and l of the same rows.
template <int D> __host__ __device__ constexpr int join_row() { return D + 4; }

template <int D> __host__ __device__ constexpr size_t smem_total() {
    return 1024 + 2 * kTile * D * 2 + (size_t)slots<D>() * slot_bytes<D>() + sizeof(Ctl);
}

// Shared-memory descriptors for the 128-byte swizzled layouts differ only in
// their low word (start address >> 4, and for MN-major operands the distance of
// the 64-column panels >> 4 in the upper half); the high word holds the 1024
// bytes between groups of 8 rows, the version and the swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t panel_bytes) {
    return ((saddr >> 4) & 0x3FFFu) | ((panel_bytes >> 4) << 16);
}

// The MMA warp stays converged, so that operands can live in uniform registers,
// and one elected lane (the same every time) issues: MMAs and the commits that
// wait for them.
// D[tmem] (+)= A[smem] * B[smem], operands by their descriptors' low words.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
        :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHi) : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]: the A operand is 128 lanes of bf16 pairs, 8
// columns per 16-wide step.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
        :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(kDescHi) : "memory");
}
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        :: "r"(smem_u32(bar)) : "memory");
}

// A whole 32-byte sector.
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t cluster_nctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};"
                 :: "r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// 128 consecutive columns of this warp's 32 TMEM lanes (one lane per thread),
// with the wait in the same statement.
__device__ __forceinline__ void tmem_ld_x128(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, "
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
          "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
          "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
          "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
          "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
          "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
          "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
          "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
          "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
        : "r"(taddr) : "memory");
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

// The items, and a CTA's work on them.
struct Walk {
    int b, hk, y;               // the item: sequence, key-value head, pair of tiles
    int turn;                   // whole items: this CTA's turn
    int x, n, c0, c1;           // the part: number x of n, steps c0 .. c1 - 1
    // of the sequence
    int t0, nq, len, pairs;
    // of the item: first token, tokens, tiles, positions of the first and last token
    int i0, n_tok, ntile, p0, p1;
    KeyBlocks kb;
    int steps;                  // kb.n, or 1 where no row sees a key (the step writes o = 0)

    __device__ __forceinline__ void seq(const AttnArgs& a, int tpt, int o0, int o1, int len_b) {
        t0 = o0;
        nq = o1 - o0;
        if (o0 < 0 || o1 < o0 || o1 > a.T || nq > a.max_q) {
            atomicCAS(a.err, 0, W4_ERR_GROUP_TOKENS);
            t0 = nq = 0;
        }
        len = len_b;
        pairs = (nq + 2 * tpt - 1) / (2 * tpt);
    }
    __device__ __forceinline__ void item(const AttnArgs& a, int tpt) {
        i0 = y * 2 * tpt;
        n_tok = min(nq - i0, 2 * tpt);
        ntile = n_tok > tpt ? 2 : 1;
        p0 = len - nq + i0;
        p1 = p0 + n_tok - 1;
        kb = key_blocks<kN>(max(p0, 0), p1, a.window, a.sinks);
        steps = max(kb.n, 1);
    }
    // item number q, in the order of the last pairs of all sequences and heads, the
    // pairs before them, and so on; false where a sequence has no such pair
    __device__ __forceinline__ bool pick(const AttnArgs& a, int tpt, int q) {
        const int bh = a.kv.batch * a.kv.heads, back = q / bh, i = q - back * bh;
        b = i / a.kv.heads;
        hk = i - b * a.kv.heads;
        seq(a, tpt, __ldg(a.goff + b), __ldg(a.goff + b + 1), kv_length(a.kv, b, a.max_len, a.err));
        y = pairs - 1 - back;
        if (y < 0) return false;
        item(a, tpt);
        return true;
    }
    // whole items: the one of this turn or a later one; false when there is none
    __device__ __forceinline__ bool settle(const AttnArgs& a, int tpt) {
        const int G = (int)gridDim.x;
        const int items = (a.max_q + 2 * tpt - 1) / (2 * tpt) * a.kv.batch * a.kv.heads;
        for (; turn * G < items; ++turn) {
            const int q = turn * G + ((turn & 1) ? G - 1 - (int)blockIdx.x : (int)blockIdx.x);
            if (q >= items || !pick(a, tpt, q)) continue;
            x = c0 = 0;
            n = 1;
            c1 = steps;
            return true;
        }
        return false;
    }
    template <bool SPLIT>
    __device__ __forceinline__ bool next(const AttnArgs& a, int tpt) {
        if (SPLIT) return false;            // one item per cluster
        ++turn;
        return settle(a, tpt);
    }
    // steps of tile i: tile A ends where its own last token does
    __device__ __forceinline__ int tile_steps(int i, int tpt) const {
        if (i == ntile - 1) return kb.n;
        const int q = p0 + tpt - 1;
        if (q < 0) return 0;
        const int blk = q / kN;
        return blk < kb.ns ? blk + 1 : kb.ns + max(blk - kb.w0 + 1, 0);
    }
    // first step of part i when an item's steps are cut into n runs equal to one
    __device__ __forceinline__ int cut(int i) const {
        const int each = steps / n, rest = steps - each * n;
        return i * each + min(i, rest);
    }
};

// Every row of the tokens at p0 .. p1 sees all of block j0.
__device__ __forceinline__ bool all_see(const AttnArgs& a, int j0, int p0, int p1) {
    return j0 + kN - 1 <= p0 && (a.window == 0 || p1 - j0 < a.window || j0 + kN <= a.sinks);
}

// The slots lo .. hi - 1 of such a block that no row's causal mask or window hides.
__device__ __forceinline__ void seen_slots(const AttnArgs& a, int j0, int p0, int p1, int* lo, int* hi) {
    *hi = min(max(p0 + 1 - j0, 0), kN);
    *lo = a.window ? min(max(p1 - a.window + 1 - j0, 0), *hi) : 0;
}

__device__ __forceinline__ bool non_finite(uint32_t bf16_bits) { return (bf16_bits & 0x7F80u) == 0x7F80u; }

// Adds to a finished row of o the values that the V release took out of blocks
// c0 .. c1 - 1 and that the row's token, at position p, sees: a weight is positive,
// so an infinity or NaN reaches the sum as it is.  A warp's rows have the item's
// sequence and key-value head in common, so its lanes look through the slots together
// (the few blocks with hidden slots, once each).  The row is out[0 .. D - 1], or, of a part
// to be joined, fp32 at shared::cluster address dst_o.
template <int D>
__device__ __noinline__ void add_non_finite(const AttnArgs& a, int b, int hk, int p0, int p1, KeyBlocks kb, int c0,
                                            int c1, int p, uint16_t* out, uint32_t dst_o) {
    const int lane = threadIdx.x & 31, lg = 31 - __clz(a.kv.page_size), first = max(p0, 0);
    for (int c = c0; c < c1; ++c) {
        const int j0 = kb(c) * kN;
        if (all_see(a, j0, p0, p1)) continue;
        int lo, hi;
        seen_slots(a, j0, p0, p1, &lo, &hi);
        for (int i0 = 0; i0 < kN * (D / 8); i0 += 32) {
            const int s = (i0 + lane) / (D / 8), j = j0 + s, d = (i0 + lane) % (D / 8) * 8;
            // taken out, and some row sees it
            const bool in = (s < lo || s >= hi) && j <= p1 &&
                            (a.window == 0 || first - j < a.window || j < a.sinks);
            uint4 u = make_uint4(0, 0, 0, 0);
            if (in)
                u = *reinterpret_cast<const uint4*>(
                    a.kv.v + page_of(a.kv, b, j >> lg, a.err) * a.kv.v_page_stride + hk * a.kv.v_head_stride +
                    (j & (a.kv.page_size - 1)) * a.kv.v_slot_stride + d);
            bool any = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) any |= non_finite((&u.x)[e]) || non_finite((&u.x)[e] >> 16);
            for (uint32_t m = __ballot_sync(0xffffffffu, any); m; m &= m - 1) {
                const int src = __ffs(m) - 1, js = __shfl_sync(0xffffffffu, j, src),
                          ds = __shfl_sync(0xffffffffu, d, src);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t w = __shfl_sync(0xffffffffu, (&u.x)[e >> 1], src), bits = e & 1 ? w >> 16 : w & 0xFFFFu;
                    if (!non_finite(bits) || !key_visible(js, p, a.window, a.sinks)) continue;
                    const float x = bf16_bits_to_f32((uint16_t)bits);
                    if (dst_o) st_shared_cluster(dst_o + (ds + e) * 4, ld_shared_cluster(dst_o + (ds + e) * 4) + x);
                    else out[ds + e] = f32_to_bf16_bits(bf16_bits_to_f32(out[ds + e]) + x);
                }
            }
        }
    }
}

// Zeros in place of the non-finite values in slots 0 .. lo - 1 and hi .. kN - 1 of a V
// block: 16-byte pieces t, t + 64, ...  Within the check that finds them it costs
// every call 1.2 us, inlined behind it 0.8 (2048 tokens).
template <int D>
__device__ __noinline__ void take_out(uint8_t* v, int t, int lo, int hi) {
    for (int panel = 0; panel < D / 64; ++panel)
        for (int s = 0; s < 2; ++s)
            for (int i = 8 * (s ? hi : 0) + t; i < 8 * (s ? kN : lo); i += 64) {
                uint4* p = reinterpret_cast<uint4*>(v + panel * kN * 128) + i;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t& z = (&p->x)[e];
                    z &= (non_finite(z) ? 0xFFFF0000u : ~0u) & (non_finite(z >> 16) ? 0x0000FFFFu : ~0u);
                }
            }
}

// SPLIT: the CTAs of a cluster share the steps of one item.
template <int D, bool SPLIT>
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

    if (threadIdx.x == 0) {
        mbar_init(&ctl->qfull, 1);
        mbar_init(&ctl->qempty, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
            mbar_init(&ctl->vready[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->sfull[i], 1);
            mbar_init(&ctl->pready[i][0], 4);
            mbar_init(&ctl->pready[i][1], 4);
            mbar_init(&ctl->ofull[i], 1);
            mbar_init(&ctl->oempty[i], 4);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = ctl->bad[0] = ctl->bad[1] = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) { tma_prefetch_desc(&tmQ); tma_prefetch_desc(&tmK); tma_prefetch_desc(&tmV); }
    if (warp == 9) { tmem_alloc(&ctl->tmem, 512); tmem_relinquish(); }
    pdl_wait();
    pdl_launch();

    // ---- this CTA's work (every thread finds it by itself)
    const int Hkv = a.kv.heads, nc = SPLIT ? (int)cluster_nctas() : 1;
    Walk w0;
    bool mine;
    if constexpr (SPLIT) {
        mine = w0.pick(a, tpt, (int)blockIdx.x / nc);
        w0.x = (int)cluster_ctarank();
        w0.n = nc;
        w0.c0 = mine ? w0.cut(w0.x) : 0;
        w0.c1 = mine ? w0.cut(w0.x + 1) : 0;
    } else {
        w0.turn = 0;
        mine = w0.settle(a, tpt);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    auto s_col = [&](int x) { return tmem + (uint32_t)(x * kN); };
    auto o_col = [&](int x) { return tmem + (uint32_t)(2 * kN + x * D); };
    volatile int* abort = &ctl->abort;
    // the join: row rr of this CTA's share, from part x of a tile
    const int per = kTile / nc;
    auto join_o = [&](int i, int x, int rr) {
        return reinterpret_cast<float*>(qs) + (i * kTile + x * per + rr) * join_row<D>();
    };
    auto join_ml = [&](int i, int x, int rr) {
        return reinterpret_cast<float*>(qs) + 2 * kTile * join_row<D>() + (i * kTile + x * per + rr) * 2;
    };
    const bool joins = SPLIT && mine && w0.kb.n > 0;      // the same in all CTAs of a cluster
    // the registers of 384 threads x 168: two softmax groups of 208, one of 88
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8) {
            // -------------------------------------------------------- TMA
            const int lg = 31 - __clz(a.kv.page_size);
            const int R = min(a.kv.page_size, kN), npg = kN / R, g = a.Hq / Hkv;
            uint32_t it = 0, part = 0;
            bool ok = true;
            Walk w = w0;
            for (bool go = mine; go && ok; go = w.next<SPLIT>(a, tpt)) {
                if (w.kb.n == 0 || w.c0 == w.c1) continue;
                const int c0 = w.c0, c1 = w.c1;
                // Q of the part before is no longer read
                if (part > 0) ok = __all_sync(0xffffffffu, mbar_wait(&ctl->qempty, (part - 1) & 1, abort, a.err));
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&ctl->qfull, (uint32_t)(w.ntile * tpt * g * D * 2));
                    for (int x = 0; x < w.ntile; ++x)
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d(qs + (x * (D / 64) + c) * kTile * 128, &tmQ, c * 64, w.hk * g,
                                        w.t0 + w.i0 + x * tpt, &ctl->qfull);
                }
                __syncwarp();
                ++part;
                for (int c = c0; c < c1 && ok; ++c) {
                    const int j0 = w.kb(c) * kN;
                    // lane: page pg of the block, 64-column panel pn; a page of which no row sees a
                    // key is not looked up (it may be gone) and loaded from out of bounds, as zeros
                    const int pg = lane % npg, pn = lane / npg, jp = j0 + pg * R;
                    const bool seen = jp <= w.p1 && (a.window == 0 || max(w.p0, 0) - (jp + R - 1) < a.window ||
                                                     jp < a.sinks);
                    int page = a.kv.pages;
                    if (pn < D / 64 && seen) page = page_of(a.kv, w.b, jp >> lg, a.err);
                    for (int kv = 0; kv < 2 && ok; ++kv, ++it) {
                        const int st = it % NS;
                        if (it >= (uint32_t)NS)
                            ok = __all_sync(0xffffffffu, mbar_wait(&ctl->empty[st], ((it / NS) & 1) ^ 1, abort, a.err));
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], SB);
                        __syncwarp();
                        if (pn < D / 64)
                            tma_load_4d(ring + st * SB + pn * kN * 128 + pg * R * 128, kv ? &tmV : &tmK, pn * 64,
                                        jp & (a.kv.page_size - 1), w.hk, page, &ctl->full[st]);
                    }
                }
            }
            if (lane == 0) {                              // every copy lands before the CTA ends
                if (part > 0) mbar_wait_drain(&ctl->qfull, (part - 1) & 1, a.err);
                for (uint32_t j = it > (uint32_t)NS ? it - NS : 0; j < it; ++j)
                    mbar_wait_drain(&ctl->full[j % NS], (j / NS) & 1, a.err);
            }
        } else if (warp == 9) {
            // -------------------------------------------------------- MMA
            {
                auto wait = [&](uint64_t* bar, uint32_t parity) {
                    return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, abort, a.err));
                };
                const uint32_t q_lo = desc_k(smem_u32(qs)), k_lo = desc_k(smem_u32(ring));
                const uint32_t v_lo = desc_mn(smem_u32(ring), kN * 128);
                auto mma_s = [&](int x, int st) {         // S_x = Q_x K^T
                    const uint32_t q = q_lo + x * (kTile * D * 2 >> 4), k = k_lo + st * (SB >> 4);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t off = ((i >> 2) * kTile * 128 + (i & 3) * 32) >> 4;
                        mma_ss(s_col(x), q + off, k + off, IDESC_S, i > 0);
                    }
                };
                auto mma_o = [&](int x, int st, int half, uint32_t acc) {   // O_x += P_x V over 64 keys
                    const uint32_t v = v_lo + st * (SB >> 4) + half * (4 * 2048 >> 4);
                    const uint32_t p = s_col(x) + 32 * half;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_ts(o_col(x), p + 8 * i, v + i * (2048 >> 4), IDESC_O, i > 0 ? 1u : acc);
                };
                uint32_t step = 0, part = 0;              // steps and parts of this CTA so far
                uint32_t np[2] = {0, 0}, no[2] = {0, 0};  // steps, parts by tile
                bool ok = true;
                Walk w = w0;
                for (bool go = mine; go && ok; go = w.next<SPLIT>(a, tpt)) {
                    if (w.kb.n == 0 || w.c0 == w.c1) continue;
                    const int c0 = w.c0, c1 = w.c1;
                    int end[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) end[x] = x < w.ntile ? min(w.tile_steps(x, tpt), c1) : 0;
                    const int ntile = w.ntile;
                    {
                        const uint32_t ik = 2 * step;
                        ok = wait(&ctl->qfull, part & 1) &&
                             wait(&ctl->full[ik % NS], (ik / NS) & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (c0 < end[x]) { mma_s(x, ik % NS); commit_elected(&ctl->sfull[x]); }
                        commit_elected(&ctl->empty[ik % NS]);
                        if (c0 + 1 == c1) commit_elected(&ctl->qempty);
                    }
                    for (int c = c0; c < c1 && ok; ++c, ++step) {
                        const uint32_t iv = 2 * step + 1, ik = 2 * step + 2;    // ring items of V c and K c + 1
                        const int sv = iv % NS, sk = ik % NS;
                        bool v_here = false, k_here = false;
                        auto next_s = [&](int x) {        // S_x of step c + 1
                            if (!k_here) ok = wait(&ctl->full[sk], (ik / NS) & 1);
                            if (!ok) return;
                            k_here = true;
                            tc_fence_after();
                            mma_s(x, sk);
                            commit_elected(&ctl->sfull[x]);
                            if (x == ntile - 1) {
                                commit_elected(&ctl->empty[sk]);
                                if (c + 2 == c1) commit_elected(&ctl->qempty);
                            }
                        };
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (!ok || c >= end[x]) continue;
                            if (c == c0 && no[x] > 0)     // O of this tile's part before is read
                                ok = wait(&ctl->oempty[x], (no[x] - 1) & 1);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                if (!ok) break;
                                ok = wait(&ctl->pready[x][half], np[x] & 1) &&
                                     (v_here || wait(&ctl->vready[sv], (iv / NS) & 1));
                                if (!ok) break;
                                v_here = true;
                                tc_fence_after();
                                mma_o(x, sv, half, half || c > c0);
                            }
                            if (!ok) continue;
                            ++np[x];
                            if (x == ntile - 1) commit_elected(&ctl->empty[sv]);
                            if (c + 1 == end[x]) {
                                commit_elected(&ctl->ofull[x]);
                                ++no[x];
                            } else {
                                next_s(x);
                            }
                        }
                    }
                    ++part;
                }
                // every MMA completes before the CTA ends
                commit_elected(&ctl->drain);
                mbar_wait_drain(&ctl->drain, 0, a.err);
                __syncwarp();
            }
        } else {
            // -------------------------------------------------------- V release
            uint32_t step = 0, part = 0;
            bool ok = true;
            Walk w = w0;
            for (bool go = mine; go && ok; go = w.next<SPLIT>(a, tpt)) {
                if (w.kb.n == 0 || w.c0 == w.c1) continue;
                const int c0 = w.c0, c1 = w.c1;
                bool bad = false;
                for (int c = c0; c < c1; ++c, ++step) {
                    const uint32_t iv = 2 * step + 1;
                    const int st = iv % NS, j0 = w.kb(c) * kN;
                    ok = __all_sync(0xffffffffu, mbar_wait(&ctl->full[st], (iv / NS) & 1, abort, a.err));
                    if (!ok) break;
                    if (!all_see(a, j0, w.p0, w.p1)) {
                        uint8_t* v = ring + st * SB;
                        // slots that some query does not see: past the first token, or out of
                        // the last one's window
                        int lo, hi;
                        seen_slots(a, j0, w.p0, w.p1, &lo, &hi);
                        // 16-byte pieces of 128-byte rows (the swizzle only permutes a row's pieces)
                        bool found = false;
                        auto check = [&](int r0, int r1) {
                            for (int panel = 0; panel < D / 64; ++panel)
                                for (int i = 8 * r0 + (warp - 10) * 32 + lane; i < 8 * r1; i += 64) {
                                    uint4* p = reinterpret_cast<uint4*>(v + panel * kN * 128) + i;
                                    if (j0 + (i >> 3) >= w.len) {
                                        *p = make_uint4(0, 0, 0, 0);
                                        continue;
                                    }
                                    const uint4 u = *p;
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const uint32_t z = (&u.x)[e];
                                        found |= non_finite(z) || (z & 0x7F800000u) == 0x7F800000u;
                                    }
                                }
                        };
                        check(0, lo);
                        check(hi, kN);
                        if (__any_sync(0xffffffffu, found)) {
                            take_out<D>(v, (warp - 10) * 32 + lane, lo, hi);
                            bad = true;
                        }
                        fence_proxy_async_smem();
                    }
                    if (lane == 0 && bad) *(volatile int*)&ctl->bad[warp - 10] = (int)part + 1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->vready[st]);
                }
                ++part;
            }
        }
        if (joins) { cluster_sync(); cluster_sync(); }
    } else {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int tile = warp >> 2, r = threadIdx.x & 127, g = a.Hq / Hkv, rt = r / g;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = s_col(tile) + lane_base, o_addr = o_col(tile) + lane_base;
        const float sc = a.scale;
        uint32_t ns = 0, no = 0, part = 0;                // steps and parts of this tile, parts of the CTA
        bool ok = true;
        Walk w = w0;
        for (bool go = mine; go && ok; go = w.next<SPLIT>(a, tpt)) {
            const int c0 = w.c0, c1 = w.c1;
            const int bad_at = (int)part;
            if (w.kb.n > 0 && c0 < c1) ++part;
            // row r of tile x: token i0 + x tpt + r / g, query head hk g + r % g
            const int tok_in = tile * tpt + rt;
            const bool have = rt < tpt && tok_in < w.n_tok;
            const int tok = w.t0 + w.i0 + tok_in, head = w.hk * g + (r - rt * g);
            const int p = have ? w.p0 + tok_in : -1;
            const size_t row = (size_t)tok * a.Hq + head;
            const int n_steps = tile < w.ntile ? w.tile_steps(tile, tpt) : 0, end = min(n_steps, c1);
            if (!joins && end <= c0) {
                // rows that see no key (where parts are joined, the join writes them)
                if (c0 == 0 && have) {
                    for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(a.out + row * D + d) = make_uint4(0, 0, 0, 0);
                    if (a.lse) a.lse[row] = kNegInf;
                }
                continue;
            }
            float m = kNegInf, l = 0.f;
            for (int c = c0; c < end; ++c, ++ns) {
                ok = __all_sync(0xffffffffu, mbar_wait(&ctl->sfull[tile], ns & 1, abort, a.err));
                if (!ok) break;
                tc_fence_after();
                uint32_t su[kN];
                tmem_ld_x128(s_addr, su);
                float* s = reinterpret_cast<float*>(su);
                const int j0 = w.kb(c) * kN;
                if (!all_see(a, j0, w.p0, w.p1)) {
                    // bit i of a word: key 32 z + i of the block is seen
                    const int hi = p - j0, lo = a.window ? hi - a.window + 1 : 0, sk = a.sinks - j0;
                    auto below = [](int k) { return k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1u; };
#pragma unroll
                    for (int z = 0; z < kN / 32; ++z) {
                        const uint32_t see = below(hi + 1 - 32 * z) & (~below(lo - 32 * z) | below(sk - 32 * z));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(see & (1u << i))) s[32 * z + i] = kNegInf;
                    }
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < kN; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx[e] = i + 4 < kN ? fmaxf(fmaxf(mx[e], s[i + e]), s[i + 4 + e]) : fmaxf(mx[e], s[i + e]);
                const float mn = fmaxf(fmaxf(m, mx[0]), fmaxf(fmaxf(mx[1], mx[2]), mx[3]));
                // S complete means this tile's O of the step before is complete too
                // rows without a query hold what was there before: they have no say, or the
                // same inputs would not give the same bits
                if (__any_sync(0xffffffffu, have && (mn - m) * sc > kLazy)) {
                    const float f = mn == m ? 1.f : ex2_approx((m - mn) * sc);
                    m = mn;
                    l *= f;
                    if (c > c0) {
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
                    if (i & 1) {                          // 64 keys of P: the MMAs may take them
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl->pready[tile][i >> 1]);
                    }
                }
                float x, z;
                unpack2(add2(sum[0], sum[1]), &x, &z);
                l += x + z;
            }
            // -------------------------------------------------------- O to memory
            const bool act = c0 < end;
            if (act) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl->ofull[tile], no & 1, abort, a.err));
                ++no;
                tc_fence_after();
            }
            // a part's row goes to the CTA that joins it
            uint32_t dst_o = 0, dst_ml = 0;
            if (joins) {
                dst_o = mapa_shared(smem_u32(join_o(tile, w.x, r % per)), r / per);
                dst_ml = mapa_shared(smem_u32(join_ml(tile, w.x, r % per)), r / per);
                cluster_sync();             // every CTA is done with its Q and its ring
            }
            if (act && ok) {
                const bool bad = __any_sync(
                    0xffffffffu, max(((volatile int*)ctl->bad)[0], ((volatile int*)ctl->bad)[1]) > bad_at);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                // rows lie apart, so a store is one sector a lane: whole sectors where `out` allows
                const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(o_addr + 32 * i, o);
                    if (!have) continue;
                    if (SPLIT) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            st_cluster_v4(dst_o + (32 * i + e) * 4, o[e], o[e + 1], o[e + 2], o[e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            uint32_t q[8];
#pragma unroll
                            for (int z = 0; z < 8; ++z)
                                q[z] = pack_bf16x2(__uint_as_float(o[e + 2 * z]) * inv, __uint_as_float(o[e + 2 * z + 1]) * inv);
                            uint16_t* to = a.out + row * D + 32 * i + e;
                            if (wide) {
                                st_global_v8(to, q);
                            } else {
                                reinterpret_cast<uint4*>(to)[0] = make_uint4(q[0], q[1], q[2], q[3]);
                                reinterpret_cast<uint4*>(to)[1] = make_uint4(q[4], q[5], q[6], q[7]);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->oempty[tile]);      // O may be overwritten
                if (bad)
                    add_non_finite<D>(a, w.b, w.hk, w.p0, w.p1, w.kb, c0, end, p, a.out + row * D, dst_o);
                if (SPLIT) {
                    st_shared_cluster(dst_ml, m);
                    st_shared_cluster(dst_ml + 4, l);
                } else if (have && a.lse) {
                    a.lse[row] = l == 0.f ? kNegInf : (m * sc + log2f(l)) * 0.6931471805599453f;
                }
            }
            if (joins) {
                cluster_sync();             // every part's rows have arrived
                // eight threads a row of this CTA's share
                constexpr int C = D / 8;
                for (int i = threadIdx.x / 8; i < w.ntile * per && ok; i += 32) {
                    const int jt = i / per, rr = i - jt * per, R = w.x * per + rr, t_in = R / g, d = (threadIdx.x & 7) * C;
                    if (t_in >= tpt || jt * tpt + t_in >= w.n_tok) continue;
                    const size_t out_row = (size_t)(w.t0 + w.i0 + jt * tpt + t_in) * a.Hq + w.hk * g + (R - t_in * g);
                    const int steps = w.tile_steps(jt, tpt);
                    float mt = kNegInf, lt = 0.f, v[C];
#pragma unroll
                    for (int e = 0; e < C; ++e) v[e] = 0.f;
                    for (int x = 0; x < nc && w.cut(x) < steps; ++x) mt = fmaxf(mt, join_ml(jt, x, rr)[0]);
                    for (int x = 0; x < nc && w.cut(x) < steps; ++x) {
                        const float mi = join_ml(jt, x, rr)[0], f = mi == mt ? 1.f : ex2_approx((mi - mt) * sc);
                        lt += f * join_ml(jt, x, rr)[1];
#pragma unroll
                        for (int e = 0; e < C; e += 4) {
                            const float4 q = *reinterpret_cast<const float4*>(join_o(jt, x, rr) + d + e);
                            v[e] += f * q.x; v[e + 1] += f * q.y; v[e + 2] += f * q.z; v[e + 3] += f * q.w;
                        }
                    }
                    const float it = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
                    for (int e = 0; e < C; e += 8)
                        *reinterpret_cast<uint4*>(a.out + out_row * D + d + e) =
                            make_uint4(pack_bf16x2(v[e] * it, v[e + 1] * it), pack_bf16x2(v[e + 2] * it, v[e + 3] * it),
                                       pack_bf16x2(v[e + 4] * it, v[e + 5] * it), pack_bf16x2(v[e + 6] * it, v[e + 7] * it));
                    if (a.lse && d == 0)
                        a.lse[out_row] = lt == 0.f ? kNegInf : (mt * sc + log2f(lt)) * 0.6931471805599453f;
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D>
int go(const AttnArgs& a, int sm_count, cudaStream_t stream) {
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
    auto encode = [](CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box) {
        return encode_tmap_nd(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rank, dims, strides, box,
                              CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!encode(&tmQ, a.q, 3, qd, qst, qb) || !encode(&tmK, a.kv.k, 4, kd, ks, kbx) ||
        !encode(&tmV, a.kv.v, 4, kd, vs, kbx))
        return W4_ERR_CUDA;
    const long long items = ((long long)a.max_q + 2 * tpt - 1) / (2 * tpt) * a.kv.heads * a.kv.batch;
    if (items > (1LL << 26)) return W4_ERR_UNSUPPORTED_SHAPE;
    // CTAs of a cluster that share an item: the fewest with the shortest last turn,
    // from upper bounds of the items and of an item's steps.  In units of a step
    // (1.8 us for heads of 128), starting and finishing an item costs about 3, with
    // the join of its parts 5.  On 1, 2, 4, 8 CTAs an item (28 / 4 heads of 128):
    // 16 tokens behind 8176 take 86.9, 52.2, 31.3, 21.0 us, 2048 behind 14336 393,
    // 345, 453, 647, twice 300 behind 3796 59, 42, 59, 107, eight prompts of 512
    // tokens 41, 105, 206, 452; the rule takes the best of each.
    const long long cap = std::min((long long)a.kv.max_pages * a.kv.page_size, (long long)a.max_len);
    long long keys = cap;
    if (a.window) keys = std::min(cap, (long long)a.window + 2 * tpt + kN + std::min<long long>(a.sinks, cap));
    const long long steps = std::max((keys + kN - 1) / kN, 1LL);
    int nc = 1;
    long long best = (items + sm_count - 1) / sm_count * (steps + 3);
    for (int c = 2; c <= 8; c *= 2) {
        const long long cost = (items * c + sm_count - 1) / sm_count * ((steps + c - 1) / c + 5);
        if (cost < best) { best = cost; nc = c; }
    }
    constexpr size_t bytes = smem_total<D>();
    auto kern = nc > 1 ? k_attn_prefill<D, true> : k_attn_prefill<D, false>;
    static SmemLimit limit[2];
    if (!limit[nc > 1].raise(kern, (int)bytes)) return W4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(nc > 1 ? items * nc : std::min<long long>(items, sm_count)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)nc;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = nc > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, tmQ, tmK, tmV, a, tpt) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

}  // namespace

int launch_attn_prefill(const AttnArgs& a, int sm_count, cudaStream_t stream) {
    return a.kv.head_dim == 128 ? go<128>(a, sm_count, stream) : go<64>(a, sm_count, stream);
}

}  // namespace w4
