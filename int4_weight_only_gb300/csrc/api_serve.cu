// api_serve.cu - the extern "C" entry points of expert routing and page plans (declared in
// include/w4.h): argument checks on the host, then the launches.
#include "w4_internal.h"

#include <algorithm>
#include <cmath>

namespace w4 {
namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// What gather and combine have in common.
int check_move(const uint16_t* x, const int32_t* row, const uint16_t* out, int T, int k, int K, int R) {
    if (T < 0 || k < 1 || K < 1 || R < 0) return W4_ERR_INVALID_ARG;
    if (k > W4_MOE_MAX_TOPK || K > (1 << 22)) return W4_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return W4_OK;
    if (!x || !row || !out) return W4_ERR_NULL_PTR;
    if (!aligned(x, 2) || !aligned(out, 2) || !aligned(row, 4)) return W4_ERR_MISALIGNED;
    return W4_OK;
}

}  // namespace
}  // namespace w4

using namespace w4;

extern "C" {

int w4_kv_plan(const int32_t* lens, const int32_t* new_tokens, const int32_t* free_pages, int n_free,
               const int32_t* used, int32_t* table, long long table_stride, int batch, int max_pages, int page_size,
               int pages, int T, int32_t* kv_len, int32_t* goff, int32_t* pos, int64_t* slots, int32_t* lens_out,
               int32_t* used_out, void* stream) {
    if (batch < 0 || T < 0 || n_free < 0 || max_pages < 1 || pages < 1 || table_stride < 0) return W4_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 4096 || (page_size & (page_size - 1)) || batch > W4_KV_PLAN_MAX_BATCH ||
        T > (1 << 30) || n_free > (1 << 30) || (long long)max_pages * page_size > (1LL << 30))
        return W4_ERR_UNSUPPORTED_SHAPE;
    if (batch > 1 && table_stride < max_pages) return W4_ERR_INVALID_ARG;      // rows would overlap
    if (!used || !goff || (batch > 0 && (!lens || !table || !kv_len)) || (T > 0 && (!pos || !slots)) ||
        (n_free > 0 && !free_pages))
        return W4_ERR_NULL_PTR;
    for (const void* p : {(const void*)lens, (const void*)new_tokens, (const void*)free_pages, (const void*)used,
                          (const void*)table, (const void*)kv_len, (const void*)goff, (const void*)pos,
                          (const void*)lens_out, (const void*)used_out})
        if (!aligned(p, 4)) return W4_ERR_MISALIGNED;
    if (!aligned(slots, 8)) return W4_ERR_MISALIGNED;
    PlanArgs a{};
    a.lens = lens; a.fresh = new_tokens; a.free_pages = free_pages; a.used = used;
    a.table = table; a.table_stride = table_stride;
    a.n_free = n_free; a.batch = batch; a.max_pages = max_pages; a.page_size = page_size; a.pages = pages; a.T = T;
    a.kv_len = kv_len; a.goff = goff; a.pos = pos; a.slots = slots; a.lens_out = lens_out; a.used_out = used_out;
    a.in_place = (lens_out && lens_out == lens) || (used_out && used_out == used);
    a.err = device_error_flag();
    if (!a.err) return W4_ERR_CUDA;
    return launch_kv_plan(a, static_cast<cudaStream_t>(stream));
}

size_t w4_moe_route_workspace_bytes(int T, int E) {
    if (T <= kRouteOne || E < 1 || E > W4_MOE_MAX_EXPERTS) return 0;
    return (size_t)route_blocks(T) * route_pitch(E) * sizeof(uint16_t);
}

int w4_moe_route(const void* logits, int logits_bf16, long long logits_stride, const float* bias, const int32_t* count,
                 int T, int E, int k, int score, int groups, int top_groups, int group_best, int renorm, float scale,
                 float* weights, int32_t* ids, int32_t* row, int32_t* goff, void* workspace, size_t workspace_bytes,
                 void* stream) {
    if (T < 0 || E < 1 || k < 1 || k > E || groups < 1 || E % groups || top_groups < 1 || top_groups > groups ||
        (long long)k > (long long)top_groups * (E / groups) || group_best < 1 || group_best > 2 ||
        (score != W4_MOE_SOFTMAX && score != W4_MOE_SIGMOID) || logits_stride < 0 || !std::isfinite(scale))
        return W4_ERR_INVALID_ARG;
    if (E > W4_MOE_MAX_EXPERTS || k > W4_MOE_MAX_TOPK || groups > 32 || T > (1 << 22) || (long long)T * k > 0x7fffffff)
        return W4_ERR_UNSUPPORTED_SHAPE;
    if (!goff || (T > 0 && (!logits || !weights || !ids || !row))) return W4_ERR_NULL_PTR;
    if (!aligned(logits, logits_bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(count, 4) || !aligned(weights, 4) ||
        !aligned(ids, 4) || !aligned(row, 4) || !aligned(goff, 4))
        return W4_ERR_MISALIGNED;
    const size_t need = w4_moe_route_workspace_bytes(T, E);
    if (need && (!workspace || workspace_bytes < need)) return W4_ERR_WORKSPACE;
    if (need && !aligned(workspace, 16)) return W4_ERR_MISALIGNED;
    RouteArgs a{};
    a.logits = logits; a.stride = logits_stride; a.bias = bias; a.count = count;
    a.bf16 = logits_bf16 ? 1 : 0;
    a.T = T; a.E = E; a.k = k; a.sigmoid = score == W4_MOE_SIGMOID;
    a.groups = groups; a.gsize = E / groups; a.top_groups = top_groups; a.best = group_best;
    a.renorm = renorm ? 1 : 0; a.scale = scale;
    a.lanes = 32;
    while (a.lanes * groups > 32) a.lanes /= 2;
    a.group_inv = ((1 << 20) + a.gsize - 1) / a.gsize;
    a.weights = weights; a.ids = ids; a.row = row; a.goff = goff;
    a.hist = static_cast<uint16_t*>(workspace);
    a.pitch = route_pitch(E);
    const int blocks = std::max(route_blocks(T), 1);
    a.per = std::max((T + blocks - 1) / blocks, 1);
    return launch_moe_route(a, static_cast<cudaStream_t>(stream));
}

int w4_moe_gather(const uint16_t* x, long long x_stride, const int32_t* row, uint16_t* out, int T, int k, int K, int R,
                  void* stream) {
    // a buffer of no rows: nothing is copied, rows other than -1 are flagged
    const int rc = check_move(x, row, R == 0 && !out ? x : out, T, k, K, R);
    if (rc) return rc;
    if (x_stride < 0) return W4_ERR_INVALID_ARG;
    if (T == 0) return W4_OK;
    MoveArgs a{};
    a.x = x; a.stride = T == 1 ? 0 : x_stride; a.row = row; a.out = out;
    a.T = T; a.k = k; a.K = K; a.R = R;
    a.err = device_error_flag();
    if (!a.err) return W4_ERR_CUDA;
    return launch_moe_gather(a, static_cast<cudaStream_t>(stream));
}

int w4_moe_combine(const uint16_t* y, const int32_t* row, const float* weights, const uint16_t* shared, uint16_t* out,
                   int T, int k, int N, int R, void* stream) {
    // no expert rows at all is a call whose every row is -1: y may be NULL then
    const int rc = check_move(R == 0 && !y ? out : y, row, out, T, k, N, R);
    if (rc) return rc;
    if (T == 0) return W4_OK;
    if (!weights) return W4_ERR_NULL_PTR;
    if (!aligned(weights, 4) || !aligned(shared, 2)) return W4_ERR_MISALIGNED;
    MoveArgs a{};
    a.x = y; a.row = row; a.weights = weights; a.shared = shared; a.out = out;
    a.T = T; a.k = k; a.K = N; a.R = R;
    a.err = device_error_flag();
    if (!a.err) return W4_ERR_CUDA;
    return launch_moe_combine(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
