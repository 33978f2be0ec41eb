// moe_route.cu - the experts of every token, and the order in which the grouped
// linears take them.
//
//   p = softmax(z) or sigmoid(z),  s = p + bias,  the k largest s among the kept groups
//   w = p of the chosen, over their sum;  row = place in the order (expert, token)
//
// A warp takes a token: logit e of it sits in lane e % 32, register e / 32; the next token's
// logits are on their way meanwhile.  Each lane keeps its two best, so that a round of the
// selection is one warp reduction over the lanes' heads, and only a lane that has given
// both looks through its registers again (with 256 experts and k = 8, one token in 20).
//
// Scores closer than their fp32 errors could come out in the wrong order, and another expert
// would be chosen than the definition says.  Without a bias nothing is at stake: the logits
// have the order of the scores.  With one, the warp looks at the gaps between the chosen and
// to what is left.  Where one is closer than the errors allow (and the two experts do not have
// the same logit and bias, which is a true tie), the chosen and those as close are ranked by
// their scores in 64 bits, one candidate a lane (settle).  So are groups whose ranks are that
// close, by the experts that can be among their best (settle_groups).  A token with more
// candidates than lanes is chosen again in 64 bits altogether (choose_wide, 20 times as long).
//
// The order is a counting sort without atomics on results: in a run of 32 tokens, bit t of an
// expert's word says that token t chose it, so a choice's rank among the run's is a population
// count.  Up to kRouteOne tokens one CTA does all; above, each CTA leaves its counts by
// expert, and a second kernel's CTAs add those of all the CTAs (and of those before them).
//
// Bound by the instructions of the selection (16384 tokens of 256 experts: issue slots 72 % busy
// with 32 warps an SM, HBM under 1 %; 770 instructions a token for k = 8, 60 a round before
// the lanes kept their heads as keys, 50 since; scores and a bias add 225, groups 470).  Measured in
// a graph: 16384 x 256 22.6 us without a bias, 29.0 with, 36.4 in 8 groups ranked by two
// scores (17 MB of logits are 2.7 us); 16384 x 384 34, 45 and 59, x 1024 65, 94 and 118 (the
// registers of 512 threads an SM); 1003 x 60 9.4; 16 x 128 in one CTA 4.4.  Rows with one
// dominant score leave the others' within its errors, and more is ranked again: softmax of
// logits of deviation 3, 5 and 8 with a bias of 0.03 46, 90 and 146 us (of 1.3: 30).
#include "block_device.cuh"
#include "w4_internal.h"

#include <algorithm>

namespace w4 {
namespace {

constexpr float kInf = __builtin_huge_valf();
constexpr uint32_t kAll = 0xffffffffu;

// How far two scores of a row can be off against each other, over its largest p.  Each is off by
// the exponential's 2^-22 of p (a sigmoid: of p (1 - p) <= 1/4) and the reciprocal's 2^-23.  The
// exponential's argument is rounded to 2^-23 of its size: times p that is below 2^-24 of the largest
// p where it is a distance from the largest logit; a sigmoid of a negative logit x is off by
// 2^-23 |x| of itself, at worst that of the largest.  The roundings of a softmax's sum, over
// V registers and 5 steps, and of its reciprocal are the same for both.  The rounding of
// p + bias adds kCloseSum of the larger score.  Scores below 2^-126 are flushed to zero: kFlushed.
template <int V> __device__ __forceinline__ float close_of(bool sigmoid, float m) {
    return sigmoid ? 0x1.4p-20f + 0x1p-22f * fmaxf(-m, 0.f) : 0x1p-20f + (V + 7) * 0x1p-24f;
}
constexpr float kCloseSum = 0x1p-23f, kFlushed = 0x1p-125f;
// A group's rank is off by the errors of its scores and three roundings of 2^-24 of their sizes, of p + bias, of the
// sum and of the bounds that it is compared by (a little more: the sizes are the computed ones).  Other experts' scores
// are no part of it, or one that a bias of -1e9 switches off would make all groups look close (16384 x 256: 585 us).
constexpr float kCloseRank = 0x1.82p-23f;

// Order-preserving key of a float that is not NaN; 0 is below every key of a value over -inf.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ float warp_max(float v) {
    return value_of(__reduce_max_sync(kAll, key_of(v)));
}
__device__ __forceinline__ double warp_sum_wide(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Logit e of token t: NaN as -inf, -0 as +0 (equal values have equal bits).
__device__ __forceinline__ float clean(float v) { return fmaxf(v, -kInf) + 0.f; }
__device__ __forceinline__ float logit_of(const RouteArgs& a, int t, int e) {
    const long long at = t * a.stride + e;
    return clean(a.bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.logits)[at])
                        : static_cast<const float*>(a.logits)[at]);
}
// A lane's logits as they are, -inf past the last expert.
template <int V> __device__ __forceinline__ void load_logits(const RouteArgs& a, int t, float* x) {
    const int lane = threadIdx.x & 31;
    if (a.bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(a.logits) + t * a.stride + lane;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i * 32 + lane < a.E ? bf16_bits_to_f32(__ldg(p + i * 32)) : -kInf;
    } else {
        const float* p = static_cast<const float*>(a.logits) + t * a.stride + lane;
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i * 32 + lane < a.E ? __ldg(p + i * 32) : -kInf;
    }
}

// p of logit x, given the row's largest logit and sum of exponentials over it.
__device__ __forceinline__ float soft_num(float x, float m) { return m == kInf ? (x == kInf ? 1.f : 0.f) : expf(x - m); }
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + expf(-x)); }
// The same for comparisons, by the hardware's 2^x (2^-22) and reciprocal (2^-23).
constexpr float kLog2e = 1.4426950408889634f;                  // (softmax weights not renormalised, whose
                                                              // sum is of these: 1.2e-7 off in the norm)
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_sigmoid(float x) { return rcp_approx(1.f + ex2_approx(-kLog2e * x)); }
__device__ __forceinline__ double soft_num(double x, double m) { return isinf(m) && m > 0 ? (x == m ? 1. : 0.) : exp(x - m); }
__device__ __forceinline__ double sigmoid(double x) { return 1. / (1. + exp(-x)); }

// The two largest of what two lanes have, largest first.
template <typename F> __device__ __forceinline__ void top_two(F& a, F& b, F c, F d) {
    const F hi = a > c ? a : c, lo = a > c ? c : a;
    const F other = b > d ? b : d;
    a = hi;
    b = lo > other ? lo : other;
}
// What a group is ranked by; two scores by half their sum, which fp32 holds for any two.
template <typename F> __device__ __forceinline__ F group_rank(F a, F b, int best) {
    const F half = F(0.5);
    return best == 2 ? (b > -kInf ? half * a + half * b : half * a) : a;
}

// The same choice in 64 bits: lane j's expert, or -1.
template <int V>
__device__ __noinline__ int choose_wide(const RouteArgs& a, int t) {
    const int lane = threadIdx.x & 31;
    double x[V], m = -kInf, sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = i * 32 + lane < a.E ? (double)logit_of(a, t, i * 32 + lane) : -kInf;
        m = x[i] > m ? x[i] : m;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const double v = __shfl_xor_sync(kAll, m, o);
        m = v > m ? v : m;
    }
    if (!a.sigmoid) {
        for (int i = 0; i < V; ++i) sum += x[i] > -kInf ? soft_num(x[i], m) : 0.;
        sum = warp_sum_wide(sum);
    }
    // what groups are ranked by; without a bias experts are chosen by their logits
    double s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i * 32 + lane;
        double p = -kInf;
        if (x[i] > -kInf) {
            p = a.sigmoid ? sigmoid(x[i]) : soft_num(x[i], m) / sum;
            if (a.bias) p += (double)__ldg(a.bias + e);
            if (!(p > -kInf)) p = -kInf;
        }
        s[i] = p;
    }
    if (a.groups > 1) {
        double mine = -kInf;
        for (int g = 0; g < a.groups; ++g) {
            double b1 = -kInf, b2 = -kInf;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if ((i * 32 + lane) / a.gsize == g) top_two<double>(b1, b2, s[i], -kInf);
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const double c1 = __shfl_xor_sync(kAll, b1, o), c2 = __shfl_xor_sync(kAll, b2, o);
                top_two(b1, b2, c1, c2);
            }
            if (lane == g) mine = group_rank(b1, b2, a.best);
        }
        int above = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double v = __shfl_sync(kAll, mine, g);
            above += v > mine || (v == mine && g < lane);
        }
        const uint32_t keep = __ballot_sync(kAll, lane < a.groups && above < a.top_groups);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * 32 + lane < a.E && !(keep >> ((i * 32 + lane) / a.gsize) & 1)) s[i] = -kInf;
    }
    if (!a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = s[i] > -kInf ? x[i] : -kInf;
    }
    int id = -1;
    for (int j = 0; j < a.k; ++j) {
        double best = -kInf;
        int at = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (s[i] > best) { best = s[i]; at = i * 32 + lane; }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const double v = __shfl_xor_sync(kAll, best, o);
            const int w = __shfl_xor_sync(kAll, at, o);
            if (v > best || (v == best && w < at)) { best = v; at = w; }
        }
        if (at == 0x7fffffff) break;
        if (lane == j) id = at;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (at == i * 32 + lane) s[i] = -kInf;
    }
    return id;
}

// p of expert e in 64 bits, for the lanes that have one (e >= 0), plus its bias.
__device__ __forceinline__ double wide_score(const RouteArgs& a, int t, int e, float m) {
    double sum = 1.;
    if (!a.sigmoid) {
        sum = 0.;
#pragma unroll 1
        for (int i = threadIdx.x & 31; i < a.E; i += 32) {
            const float x = logit_of(a, t, i);
            sum += x > -kInf ? soft_num((double)x, (double)m) : 0.;
        }
        sum = warp_sum_wide(sum);
    }
    if (e < 0) return -kInf;
    const double x = logit_of(a, t, e), p = a.sigmoid ? sigmoid(x) : soft_num(x, (double)m) / sum;
    return a.bias ? p + (double)__ldg(a.bias + e) : p;
}

// Ranks the n <= 32 candidates of token t, one a lane (e < 0: none), by their scores in 64 bits;
// returns the one of rank `lane`.  m: the row's largest logit.
__device__ __noinline__ int settle(const RouteArgs& a, int t, int e, int n, float m) {
    const int lane = threadIdx.x & 31;
    const double s = wide_score(a, t, e, m);
    int rank = 0, got = -1;
#pragma unroll 1
    for (int o = 0; o < n; ++o) {
        const double v = __shfl_sync(kAll, s, o);
        const int w = __shfl_sync(kAll, e, o);
        rank += w >= 0 && (v > s || (v == s && w < e));
    }
#pragma unroll 1
    for (int o = 0; o < n; ++o) {
        const int w = __shfl_sync(kAll, e, o), r = __shfl_sync(kAll, rank, o);
        if (w >= 0 && r == lane) got = w;
    }
    return got;
}

// Every expert offered to token t has the same logit and bias (a padded row's, say): ties between groups that rank by
// as many scores are true ones.  m: the largest logit.
__device__ __noinline__ bool all_alike(const RouteArgs& a, int t, const float* bias, float m) {
    const int lane = threadIdx.x & 31;
    float b = -kInf;
    if (a.bias)
        for (int e = lane; e < a.E; e += 32) b = fmaxf(b, bias[e]);
    b = warp_max(b);
    bool same = true;
    for (int e = lane; e < a.E; e += 32) {
        const float x = logit_of(a, t, e);
        if (x > -kInf && !(a.bias && bias[e] == -kInf)) same &= x == m && (!a.bias || bias[e] == b);
    }
    return __all_sync(kAll, same);
}

// Whether a lane's group is kept, where ranks lie within their errors of the border: low, high, the least and the most
// that the group's exact rank can be; kept, what the computed ranks say.  A kept group above all that are not (hi, the
// most of theirs) stays, one that is below all the kept (lo, the least of theirs) goes; the others are ranked in 64
// bits by those of their experts that can be among the best (buf from `from` on).  False in *fits: more candidates
// than lanes.
template <int V>
__device__ __noinline__ bool settle_groups(const RouteArgs& a, int t, const float* buf, bool kept, float low, float high,
                                           float from, float lo, float hi, float m, bool* fits) {
    const int lane = threadIdx.x & 31, L = a.lanes, g = lane / L;
    const bool clear = kept && low > hi, open = g < a.groups && !clear && high >= lo;
    const int left = a.top_groups - __popc(__ballot_sync(kAll, clear && lane == g * L));
    int n = 0, cand = -1, its = -1;
#pragma unroll 1
    for (int i = 0; i < V && n <= 32; ++i) {
        const int e = i * 32 + lane, ge = e < a.E ? e * a.group_inv >> 20 : 0;
        const bool o = __shfl_sync(kAll, open, ge * L);
        const float b = __shfl_sync(kAll, from, ge * L);
        const bool in = e < a.E && o && buf[e] > -kInf && !(buf[e] < b);
        for (uint32_t w = __ballot_sync(kAll, in); w; w &= w - 1, ++n)
            if (lane == n) cand = i * 32 + __ffs(w) - 1;
    }
    *fits = n <= 32;
    if (n > 32) return false;
    if (cand >= 0) its = cand * a.group_inv >> 20;
    const double s = wide_score(a, t, cand, m);
    double b1 = -kInf, b2 = -kInf;
#pragma unroll 1
    for (int o = 0; o < n; ++o) {
        const double v = __shfl_sync(kAll, s, o);
        if (__shfl_sync(kAll, its, o) == g) top_two<double>(b1, b2, v, -kInf);
    }
    const double rank = group_rank(b1, b2, a.best);
    int above = 0;
#pragma unroll 1
    for (int i = 0; i < a.groups; ++i) {
        const double v = __shfl_sync(kAll, rank, i * L);
        if (__shfl_sync(kAll, open, i * L)) above += v > rank || (v == rank && i < g);
    }
    return clear || (open && above < left);
}

// Keys of the best two of a lane's values, in the order of falling values and rising registers, 0
// where there is none; AFTER: of those behind (v0, i0).
template <int V, bool AFTER>
__device__ __forceinline__ void best_two(const float* s, float v0, int i0, uint32_t* k1, int* i1, uint32_t* k2, int* i2) {
    float b1 = -kInf, b2 = -kInf;
    *i1 = *i2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float v = !AFTER || s[i] < v0 || (s[i] == v0 && i > i0) ? s[i] : -kInf;
        const bool first = v > b1, second = v > b2;
        *i2 = first ? *i1 : second ? i : *i2;
        b2 = fmaxf(b2, fminf(b1, v));
        *i1 = first ? i : *i1;
        b1 = fmaxf(b1, v);
    }
    *k1 = b1 > -kInf ? key_of(b1) : 0u;
    *k2 = b2 > -kInf ? key_of(b2) : 0u;
}

// The experts of token t, whose logits a lane has in x: lane j gets the j-th (or -1) and its
// weight.  buf: E floats of the warp's own (groups); bias: 32 V in shared memory.
template <int V>
__device__ __forceinline__ void choose(const RouteArgs& a, int t, float* x, float* buf, const float* bias, int* id_out,
                                       float* w_out) {
    const int lane = threadIdx.x & 31;
    const bool two = a.groups > 1 && a.best == 2;   // groups ranked by sums of scores
    const bool scored = a.bias || two;
    float m = -kInf, inv = 1.f;                     // softmax: largest logit, reciprocal sum
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = clean(x[i]);
        m = fmaxf(m, x[i]);
    }
    if (scored || !a.renorm) {
        m = warp_max(m);
        if (!a.sigmoid) {
            float sum = 0.f;
            if (fabsf(m) == kInf) {                 // infinite logits, or none
#pragma unroll
                for (int i = 0; i < V; ++i) sum += x[i] == kInf ? 1.f : 0.f;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) sum += ex2_approx((x[i] - m) * kLog2e);
            }
            inv = rcp_approx(warp_sum(sum));
        }
    }
    auto prob = [&](float v) { return a.sigmoid ? sigmoid(v) : soft_num(v, m) * inv; };
    // what groups are ranked by two scores of, and experts are chosen by when there is a bias
    // (s may be x)
    auto scores = [&](float* s) {
        auto put = [&](int i, float p) {
            if (a.bias) p += bias[i * 32 + lane];
            s[i] = x[i] > -kInf ? p : -kInf;
        };
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < V; ++i) put(i, fast_sigmoid(x[i]));
        } else if (fabsf(m) == kInf) {
#pragma unroll
            for (int i = 0; i < V; ++i) put(i, x[i] == kInf ? inv : 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) put(i, ex2_approx((x[i] - m) * kLog2e) * inv);
        }
    };
    // from here x is what experts are chosen by, -inf where they are not offered
    if (a.bias) scores(x);
    const float err = scored && m > -kInf ? close_of<V>(a.sigmoid, m) * prob(m) + kFlushed : 0.f;
    bool again = false;
    if (a.groups > 1) {
        if (two && !a.bias) {
            float s[V];
            scores(s);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * 32 + lane < a.E) buf[i * 32 + lane] = s[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * 32 + lane < a.E) buf[i * 32 + lane] = x[i];
        }
        __syncwarp();
        // L lanes a group, each with every L-th of its scores; groups start at different ones,
        // so that the lanes' words lie in different banks
        const int L = a.lanes, g = lane / L, sub = lane - g * L;
        float b1 = -kInf, b2 = -kInf;
        if (g < a.groups) {
            const float* mine = buf + g * a.gsize;
            int at = g * L % a.gsize / L * L + sub;  // L divides neither gsize nor this in general
#pragma unroll 4
            for (int i = sub; i < a.gsize; i += L) {
                if (at >= a.gsize) at = sub;
                const float v = mine[at];
                b2 = fmaxf(b2, fminf(b1, v));
                b1 = fmaxf(b1, v);
                at += L;
            }
        }
        for (int o = L / 2; o; o >>= 1) {
            const float c1 = __shfl_xor_sync(kAll, b1, o), c2 = __shfl_xor_sync(kAll, b2, o);
            b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
            b1 = fmaxf(b1, c1);
        }
        const float mine = group_rank(b1, b2, a.best);
        int above = 0;
#pragma unroll 4
        for (int i = 0; i < a.groups; ++i) {
            const float v = __shfl_sync(kAll, mine, i * L);
            above += v > mine || (v == mine && i < g);
        }
        bool in = g < a.groups && above < a.top_groups;
        if (scored) {
            const float size = a.best == 2 ? 0.5f * kCloseRank * fabsf(b1) + (b2 > -kInf ? 0.5f * kCloseRank * fabsf(b2) : 0.f)
                                           : kCloseRank * fabsf(b1);
            const float off = fabsf(mine) < kInf ? 0.5f * err + size : 0.f, low = mine - off, high = mine + off;
            const float lo = -warp_max(in ? -low : -kInf), hi = warp_max(g < a.groups && !in ? high : -kInf);
            // groups at the border of which some have one expert to rank by and others two
            const bool border = g < a.groups && high >= lo && low <= hi, two_of = b2 > -kInf;
            const bool mixed = a.best == 2 && __any_sync(kAll, border && two_of) && __any_sync(kAll, border && !two_of);
            if (hi > -kInf && lo <= hi && (mixed || !all_alike(a, t, bias, m))) {
                const float edge = a.best == 2 && b2 > -kInf ? b2 : b1;
                bool fits = false;
                in = settle_groups<V>(a, t, buf, in, low, high, edge - (err + kCloseRank * fabsf(edge)), lo, hi, m, &fits);
                again = !fits;
            }
        }
        const uint32_t keep = __ballot_sync(kAll, in && sub == 0);
#pragma unroll
        for (int i = 0; i < V; ++i)                 // (i * 32 + lane) / gsize, exact below 1024
            if (!(keep >> (((i * 32 + lane) * a.group_inv >> 20) * L) & 1)) x[i] = -kInf;
        __syncwarp();                               // buf is read
    }
    int id = -1;
    if (!__any_sync(kAll, again)) {
        uint32_t k1, k2, out = 0, mine_key = 0;     // the lane's best two; its last given; what it holds was chosen by
        int i1, i2, at_out = -1, chosen = 0;
        bool second = true;                         // k2 is known
        best_two<V, false>(x, 0.f, 0, &k1, &i1, &k2, &i2);
        for (; chosen < a.k; ++chosen) {
            const uint32_t best = __reduce_max_sync(kAll, k1);
            if (best == 0) break;
            const uint32_t who = __ballot_sync(kAll, k1 == best);
            int from = __ffs(who) - 1;
            if (who & (who - 1)) {                  // equal ones: the lowest expert
                const uint32_t e = __reduce_min_sync(kAll, k1 == best ? (uint32_t)(i1 * 32 + lane) : ~0u);
                from = (int)(e & 31);
            }
            const int e = __shfl_sync(kAll, i1, from) * 32 + from;
            if (lane == chosen) { id = e; mine_key = best; }
            bool look = false;
            if (lane == from) {
                out = best;
                at_out = i1;
                k1 = k2;
                i1 = i2;
                look = !second;
                second = false;
            }
            if (__any_sync(kAll, look)) {
                if (look) { best_two<V, true>(x, value_of(out), at_out, &k1, &i1, &k2, &i2); second = true; }
            }
        }
        if (a.bias && chosen > 0) {
            // each chosen one against the one before, then what is left against the last
            const float mine = id >= 0 ? value_of(mine_key) : -kInf;
            const float s1 = __shfl_up_sync(kAll, mine, 1), last = __shfl_sync(kAll, mine, chosen - 1);
            const int e1 = __shfl_up_sync(kAll, id, 1), e_last = __shfl_sync(kAll, id, chosen - 1);
            bool close = lane > 0 && id >= 0 && s1 - mine <= err + kCloseSum * fmaxf(fabsf(s1), fabsf(mine));
            const float reach = err + kCloseSum * (fabsf(last) + err);
            uint32_t left = 0;                      // registers with an expert as good as the last
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (x[i] > -kInf && (x[i] < last || (x[i] == last && i * 32 + lane > e_last)) && last - x[i] <= reach)
                    left |= 1u << i;
            if (__any_sync(kAll, close || left)) {
                auto same = [&](int e, int f) {
                    return logit_of(a, t, e) == logit_of(a, t, f) && __ldg(a.bias + e) == __ldg(a.bias + f);
                };
                if (close && same(id, e1)) close = false;
                bool open = close;
                for (uint32_t b = left; b && !open; b &= b - 1) open = !same((__ffs(b) - 1) * 32 + lane, e_last);
                if (__any_sync(kAll, open)) {
                    int n = chosen, cand = id;
#pragma unroll 1
                    for (int i = 0; i < V && n <= 32; ++i)
                        for (uint32_t b = __ballot_sync(kAll, left >> i & 1); b; b &= b - 1, ++n)
                            if (lane == n) cand = i * 32 + __ffs(b) - 1;
                    if (n > 32) again = true;
                    else id = settle(a, t, cand, n, m);
                    if (lane >= a.k) id = -1;
                }
            }
        }
    }
    if (__any_sync(kAll, again)) id = choose_wide<V>(a, t);
    // ---- weights of the chosen
    const bool have = id >= 0;
    const float z = have ? logit_of(a, t, id) : -kInf;
    float w = 0.f;
    if (a.renorm) {
        // over the largest chosen logit (sigmoid: only if all are negative), so that weights
        // that underflow together keep their ratios
        const float c = warp_max(z);
        if (have) {
            if (!a.sigmoid) w = soft_num(z, c);
            else w = c >= 0.f ? sigmoid(z) : __fdividef(expf(z - c), 1.f + expf(z));
        }
        const float total = warp_sum(w);
        w = have && total > 0.f ? __fdividef(w, total) * a.scale : 0.f;
    } else if (have) {
        w = prob(z) * a.scale;
    }
    *id_out = id;
    *w_out = w;
}

template <int V> constexpr int route_threads() { return V <= 8 ? 1024 : 512; }

// Inclusive sum over a CTA's threads; part: a word per warp.
__device__ __forceinline__ int block_scan(int v, int* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int u = lane < warps ? part[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int q = __shfl_up_sync(kAll, u, o);
            if (lane >= o) u += q;
        }
        part[lane] = u;
    }
    __syncthreads();
    if (warp) v += part[warp - 1];
    __syncthreads();
    return v;
}

// ONE: all tokens, and their order; else the CTA's tokens and its counts.
template <int V, bool ONE>
__global__ void __launch_bounds__(route_threads<V>(), 1) k_moe_route(const RouteArgs a) {
    extern __shared__ float group_buf[];
    __shared__ float bias[V * 32];
    __shared__ uint32_t bits[ONE ? kRouteOne / 32 : 1][V * 32];       // ONE: who chose; else counts
    __shared__ int base[V * 32];
    __shared__ int part[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    for (int i = tid; i < (ONE ? kRouteOne / 32 : 1) * V * 32; i += blockDim.x) (&bits[0][0])[i] = 0;
    pdl_wait();
    pdl_launch();
    // a bias that is NaN or -inf takes its expert out
    if (a.bias)
        for (int e = tid; e < V * 32; e += blockDim.x) bias[e] = e < a.E ? fmaxf(__ldg(a.bias + e), -kInf) : 0.f;
    __syncthreads();
    const int t0 = ONE ? 0 : (int)blockIdx.x * a.per, t1 = min(a.T, t0 + (ONE ? a.T : a.per));
    const int real = a.count ? min(max(__ldg(a.count), 0), a.T) : a.T;
    float x[V], nx[V];
    if (t0 + warp < min(t1, real)) load_logits<V>(a, t0 + warp, nx);
    for (int t = t0 + warp; t < t1; t += warps) {
        int id = -1;
        float w = 0.f;
        if (t < real) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = nx[i];
            if (t + warps < min(t1, real)) load_logits<V>(a, t + warps, nx);
            choose<V>(a, t, x, group_buf + warp * a.E, bias, &id, &w);
        }
        if (lane < a.k) {
            a.ids[(size_t)t * a.k + lane] = id;
            a.weights[(size_t)t * a.k + lane] = w;
            if (id >= 0) {
                if (ONE) atomicOr(&bits[t >> 5][id], 1u << (t & 31));
                else atomicAdd(&bits[0][id], 1u);
            }
        }
    }
    __syncthreads();
    if (!ONE) {
        for (int e = tid; e < a.pitch; e += blockDim.x)
            a.hist[(size_t)blockIdx.x * a.pitch + e] = e < a.E ? (uint16_t)bits[0][e] : (uint16_t)0;
        return;
    }
    // first rows of the experts
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += blockDim.x) {
        const int e = e0 + tid;
        int c = 0;
        if (e < a.E)
#pragma unroll
            for (int i = 0; i < kRouteOne / 32; ++i) c += __popc(bits[i][e]);
        const int v = block_scan(c, part);
        if (e < a.E) {
            base[e] = carry + v - c;
            a.goff[e] = carry + v - c;
            if (e == a.E - 1) a.goff[a.E] = carry + v;
        }
        carry += part[warps - 1];
        __syncthreads();
    }
    for (int i = tid; i < a.T * a.k; i += blockDim.x) {
        const int t = i / a.k, id = a.ids[i];
        int r = -1;
        if (id >= 0) {
            r = base[id];
#pragma unroll
            for (int j = 0; j < kRouteOne / 32; ++j) {
                const int d = t - 32 * j;
                if (d > 0) r += __popc(d >= 32 ? bits[j][id] : bits[j][id] & ((1u << d) - 1u));
            }
        }
        a.row[i] = r;
    }
}

// The rows of a CTA's tokens: counts of all CTAs and of those before it, then ranks in runs of
// 128 tokens, whose ids are on their way while the counts are added.
constexpr int kOrderThreads = 512, kOrderRun = 128, kOrderAhead = 2;
constexpr int kOrderSums = kOrderThreads * 8;    // a thread adds eight experts of every `rows`-th CTA
__global__ void __launch_bounds__(kOrderThreads, 1) k_moe_order(const RouteArgs a) {
    extern __shared__ int order_smem[];             // base [pitch], total [pitch], sums 2 x [rows][pitch] or bits
    __shared__ int part[32];
    int *base = order_smem, *total = base + a.pitch, *sums = total + a.pitch;
    uint32_t* bits = reinterpret_cast<uint32_t*>(sums);            // [run / 32][pitch]
    const int tid = threadIdx.x, me = blockIdx.x, B = gridDim.x;
    const int cols = a.pitch / 8, rows = min(kOrderThreads / cols, 16), c = tid % cols, r = tid / cols;
    pdl_wait();
    pdl_launch();
    const int t1 = min(a.T, (me + 1) * a.per);
    int ahead[kOrderAhead];
    {
        const int n = min(kOrderRun, t1 - me * a.per) * a.k;
#pragma unroll
        for (int i = 0; i < kOrderAhead; ++i)
            ahead[i] = tid + i * kOrderThreads < n ? a.ids[(size_t)me * a.per * a.k + tid + i * kOrderThreads] : -1;
        int all[8], before[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) all[i] = before[i] = 0;
        if (r < rows) {
#pragma unroll 4
            for (int b = r; b < B; b += rows) {
                const uint4 u = *reinterpret_cast<const uint4*>(a.hist + (size_t)b * a.pitch + c * 8);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int v = (int)((&u.x)[i >> 1] >> (16 * (i & 1)) & 0xFFFFu);
                    all[i] += v;
                    if (b < me) before[i] += v;
                }
            }
            int4* to = reinterpret_cast<int4*>(sums + r * a.pitch + c * 8);
            to[0] = make_int4(all[0], all[1], all[2], all[3]);
            to[1] = make_int4(all[4], all[5], all[6], all[7]);
            to += kOrderSums / 4;
            to[0] = make_int4(before[0], before[1], before[2], before[3]);
            to[1] = make_int4(before[4], before[5], before[6], before[7]);
        }
    }
    __syncthreads();
    for (int e = tid; e < a.pitch; e += blockDim.x) {
        int x = 0, y = 0;
        for (int i = 0; i < rows; ++i) {
            x += sums[i * a.pitch + e];
            y += sums[kOrderSums + i * a.pitch + e];
        }
        total[e] = x;
        base[e] = y;
    }
    __syncthreads();
    for (int i = tid; i < kOrderRun / 32 * a.pitch; i += blockDim.x) bits[i] = 0;
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += blockDim.x) {
        const int e = e0 + tid, c = e < a.E ? total[e] : 0, v = block_scan(c, part);
        if (e < a.E) {
            base[e] += carry + v - c;
            if (me == 0) {
                a.goff[e] = carry + v - c;
                if (e == a.E - 1) a.goff[a.E] = carry + v;
            }
        }
        carry += part[(blockDim.x >> 5) - 1];
        __syncthreads();
    }
    for (int t0 = me * a.per; t0 < t1; t0 += kOrderRun) {
        const int n = min(kOrderRun, t1 - t0) * a.k;
        const int32_t* ids = a.ids + (size_t)t0 * a.k;
        auto id_of = [&](int i) {
            if (t0 == me * a.per) {
#pragma unroll
                for (int j = 0; j < kOrderAhead; ++j)
                    if (i == tid + j * kOrderThreads) return ahead[j];
            }
            return ids[i];
        };
        for (int i = tid; i < n; i += blockDim.x) {
            const int t = i / a.k, id = id_of(i);
            if (id >= 0) atomicOr(bits + (t >> 5) * a.pitch + id, 1u << (t & 31));
        }
        __syncthreads();
        for (int i = tid; i < n; i += blockDim.x) {
            const int t = i / a.k, id = id_of(i);
            int r = -1;
            if (id >= 0) {
                r = base[id];
#pragma unroll
                for (int j = 0; j < kOrderRun / 32; ++j) {
                    const int d = t - 32 * j;
                    const uint32_t word = bits[j * a.pitch + id];
                    if (d > 0) r += __popc(d >= 32 ? word : word & ((1u << d) - 1u));
                }
            }
            a.row[(size_t)t0 * a.k + i] = r;
        }
        if (t0 + kOrderRun >= t1) break;
        __syncthreads();
        for (int e = tid; e < a.E; e += blockDim.x)
#pragma unroll
            for (int j = 0; j < kOrderRun / 32; ++j) {
                base[e] += __popc(bits[j * a.pitch + e]);
                bits[j * a.pitch + e] = 0;
            }
        __syncthreads();
    }
}

template <typename... A>
bool launch(void (*kern)(A...), int grid, int threads, size_t smem, cudaStream_t stream, const RouteArgs& a) {
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
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess;
}

template <int V>
int go(const RouteArgs& a, cudaStream_t stream) {
    const bool one = a.T <= kRouteOne;
    // no more warps than tokens
    const int tokens = one ? a.T : a.per, threads = std::min(route_threads<V>(), std::max(128, (tokens * 32 + 127) / 128 * 128));
    const size_t smem = a.groups > 1 ? (size_t)threads / 32 * a.E * sizeof(float) : 0;
    static SmemLimit limit[2];
    constexpr int most = route_threads<V>() / 32 * V * 32 * (int)sizeof(float);
    if (one) {
        if (!limit[0].raise(k_moe_route<V, true>, most)) return W4_ERR_CUDA;
        return launch(k_moe_route<V, true>, 1, threads, smem, stream, a) ? W4_OK : W4_ERR_CUDA;
    }
    if (!limit[1].raise(k_moe_route<V, false>, most)) return W4_ERR_CUDA;
    const int grid = (a.T + a.per - 1) / a.per;
    if (!launch(k_moe_route<V, false>, grid, threads, smem, stream, a)) return W4_ERR_CUDA;
    static SmemLimit order_limit;
    if (!order_limit.raise(k_moe_order, (2 * W4_MOE_MAX_EXPERTS + 2 * kOrderSums) * (int)sizeof(int))) return W4_ERR_CUDA;
    return launch(k_moe_order, grid, kOrderThreads, (2 * a.pitch + 2 * kOrderSums) * sizeof(int), stream, a)
               ? W4_OK : W4_ERR_CUDA;
}

}  // namespace

// A few tokens a CTA: warps of one SM slow each other down (1003 tokens in CTAs of 32: 10.4 us).
int route_blocks(int T) { return std::min(kRouteBlocks, (T + 7) / 8); }

int launch_moe_route(const RouteArgs& a, cudaStream_t stream) {
    return a.E <= 64 ? go<2>(a, stream) : a.E <= 128 ? go<4>(a, stream) : a.E <= 256 ? go<8>(a, stream)
         : a.E <= 512 ? go<16>(a, stream) : go<32>(a, stream);
}

}  // namespace w4
