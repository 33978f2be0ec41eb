// kv_plan.cu - page table entries, lengths, offsets and slots of a step from the requests'
// lengths.
//
// Two sums over the requests, of the new rows and of the new pages, place everything: row t
// of the step belongs to the last request whose rows begin at or before it, and new page i
// of the step to the last request whose pages do.  All in one launch: each CTA takes the sums
// for itself, in shared memory (a few thousand requests are a few rounds of a scan), then its
// share of the requests, pages and rows.  Where outputs are the inputs (lengths and pages used
// in place) the CTAs are a cluster, which meets once all have read them.  Bound by latency:
// lengths, scan, table or free list.  Measured in a graph: 256 requests of at most one token
// 3.7 us; 97 with 118k new tokens 6.0 (a row a thread at a time on a cluster of eight 14.4).
#include "block_device.cuh"
#include "w4_internal.h"

#include <algorithm>

namespace w4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kMostCtas = 64;           // each repeats the sums
constexpr uint32_t kAll = 0xffffffffu;

// Inclusive sum over the CTA, saturating at `most` (so that sums of any inputs stay in range).
__device__ __forceinline__ unsigned block_scan(unsigned v, unsigned most, unsigned* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned u = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v = min(v + u, most);
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        unsigned u = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned q = __shfl_up_sync(kAll, u, o);
            if (lane >= o) u = min(u + q, most);
        }
        part[lane] = u;
    }
    __syncthreads();
    if (warp) v = min(v + part[warp - 1], most);
    return v;
}

// The last i in [0, n) with at[i] <= v (at[0] = 0 <= v, non-decreasing).
__device__ __forceinline__ int last_at(const int* at, int n, int v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1) k_kv_plan(const PlanArgs a) {
    extern __shared__ int smem[];
    __shared__ unsigned part[32];
    __shared__ int s_end;
    const int B = a.batch;
    int *rows = smem, *pages = rows + B + 1, *old = pages + B + 1;     // first row, first new page, length before
    const int tid = threadIdx.x;
    if (tid == 0) { rows[0] = pages[0] = s_end = 0; }
    pdl_wait();
    pdl_launch();
    const int lg = 31 - __clz(a.page_size), in_page = a.page_size - 1;
    // lengths and used may be written by this call, the table is: no read-only loads of them
    const int given = __ldcg(a.used), used = min(max(given, 0), a.n_free);
    if (used != given && tid == 0) atomicCAS(a.err, 0, W4_ERR_PAGE_TABLE);
    const unsigned left = (unsigned)(a.n_free - used), T = (unsigned)a.T;
    const long long cap = (long long)a.max_pages * a.page_size;
    unsigned row0 = 0, page0 = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + tid;
        const int len = b < B ? __ldcg(a.lens + b) : 0, asked = b < B ? (a.fresh ? __ldg(a.fresh + b) : 1) : 0;
        const unsigned n = min((unsigned)max(asked, 0), T + 1);
        const unsigned r = min(row0 + block_scan(n, T + 1, part), T + 1);     // sums past T stay past it
        row0 = min(row0 + part[31], T + 1);
        __syncthreads();
        const bool sized = len >= 0 && asked >= 0 && (long long)len + asked <= cap, fits = r <= T;
        unsigned need = 0;
        if (b < B) {
            if (!sized) atomicCAS(a.err, 0, W4_ERR_PAGE_TABLE);
            else if (!fits) atomicCAS(a.err, 0, W4_ERR_GROUP_TOKENS);
            else need = (unsigned)(((len + asked + in_page) >> lg) - ((len + in_page) >> lg));
        }
        const unsigned p = min(page0 + block_scan(need, left + 1, part), left + 1);
        page0 = min(page0 + part[31], left + 1);
        __syncthreads();
        if (b < B) {
            const bool in = sized && fits && (need == 0 || p <= left);
            if (sized && fits && !in) atomicCAS(a.err, 0, W4_ERR_NO_PAGES);
            rows[b + 1] = (int)min(r, T);
            pages[b + 1] = (int)p;
            old[b] = in ? len : -1;
            if (in && need) atomicMax(&s_end, (int)p);
        }
    }
    __syncthreads();
    const int G = (int)gridDim.x, me = (int)blockIdx.x * kThreads + tid, all = G * kThreads;
    if (a.in_place && G > 1) cluster_sync();            // every CTA has read what outputs overwrite
    const int end = s_end;
    if (me == 0 && a.used_out) *a.used_out = used + end;
    for (int b = me; b <= B; b += all) {
        a.goff[b] = rows[b];
        if (b == B) break;
        const int n = rows[b + 1] - rows[b];
        const bool in = old[b] >= 0;
        a.kv_len[b] = in && n > 0 ? old[b] + n : 0;
        if (a.lens_out) {
            if (in) a.lens_out[b] = old[b] + n;
            else if (a.lens_out != a.lens) a.lens_out[b] = __ldcg(a.lens + b);
        }
    }
    for (int i = me; i < end; i += all) {
        const int b = last_at(pages, B + 1, i);
        a.table[b * a.table_stride + ((old[b] + in_page) >> lg) + (i - pages[b])] = __ldg(a.free_pages + used + i);
    }
    // a thread takes R rows in a row, which are of one request more often than not, with one
    // search; their lookups are in flight together
    const bool wide = ((reinterpret_cast<uintptr_t>(a.pos) | reinterpret_cast<uintptr_t>(a.slots)) & 15) == 0;
    for (int t0 = R * me; t0 < a.T; t0 += R * all) {
        int pos[R], page[R], b = -1;
        long long slot[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int t = t0 + i;
            pos[i] = page[i] = -1;
            if (t >= min(rows[B], a.T)) continue;
            if (b < 0 || t >= rows[b + 1]) b = last_at(rows, B + 1, t);
            if (old[b] < 0) continue;
            const int p = old[b] + t - rows[b], held = (old[b] + in_page) >> lg, j = p >> lg;
            pos[i] = p;
            page[i] = j < held ? __ldcg(a.table + b * a.table_stride + j)
                               : __ldg(a.free_pages + used + pages[b] + (j - held));
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            slot[i] = -1;
            if (pos[i] < 0) continue;
            if ((unsigned)page[i] < (unsigned)a.pages) slot[i] = (long long)page[i] * a.page_size + (pos[i] & in_page);
            else atomicCAS(a.err, 0, W4_ERR_PAGE_TABLE);
        }
        if (R == 4 && wide && t0 + R <= a.T) {
            *reinterpret_cast<int4*>(a.pos + t0) = make_int4(pos[0], pos[1 % R], pos[2 % R], pos[3 % R]);
            *reinterpret_cast<longlong2*>(a.slots + t0) = make_longlong2(slot[0], slot[1 % R]);
            *reinterpret_cast<longlong2*>(a.slots + t0 + 2) = make_longlong2(slot[2 % R], slot[3 % R]);
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (t0 + i < a.T) {
                    a.pos[t0 + i] = pos[i];
                    a.slots[t0 + i] = slot[i];
                }
        }
    }
}

}  // namespace

template <int R>
static int go(const PlanArgs& a, int ctas, cudaStream_t stream) {
    const size_t smem = (size_t)(3 * a.batch + 2) * sizeof(int);
    static SmemLimit limit;
    if (!limit.raise(k_kv_plan<R>, (3 * W4_KV_PLAN_MAX_BATCH + 2) * (int)sizeof(int))) return W4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.in_place && ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_kv_plan<R>, a) == cudaSuccess ? W4_OK : W4_ERR_CUDA;
}

int launch_kv_plan(const PlanArgs& a, cudaStream_t stream) {
    // A CTA has a row or a request for each thread, four rows where that is more than eight CTAs
    // (one launch's rows are then prompts', whose neighbours share request and page).  Outputs in
    // place of inputs need all CTAs in one cluster, eight at most (the portable size).
    const bool four = a.T > 8 * kThreads;
    const int want = (std::max(four ? a.T / 4 : a.T, a.batch) + kThreads - 1) / kThreads;
    int ctas = std::min(std::max(want, 1), kMostCtas);
    if (a.in_place) {
        ctas = 1;
        while (ctas < 8 && ctas < want) ctas *= 2;
    }
    return four ? go<4>(a, ctas, stream) : go<1>(a, ctas, stream);
}

}  // namespace w4
